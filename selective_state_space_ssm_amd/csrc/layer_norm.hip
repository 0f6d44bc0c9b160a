// layer_norm.hip -- the layer norm of the residual stream and its gradients.
//
//   s  = x + residual                     (float32; x alone without a residual)
//   mu = mean_D(s),  rs = 1 / sqrt(mean_D((s - mu)^2) + eps)
//   y  = (s - mu) * rs * w + b
// and, with xh = (s - mu) * rs and g = dy * w,
//   dx = rs * (g - mean_D(g) - xh * mean_D(g * xh))  (+ dresidual)
//   dw = sum_T dy * xh,   db = sum_T dy
//
// A row lives in the registers of the G lanes that share it (16 lanes to a
// whole workgroup), as 16-byte vectors, so memory is read and written once;
// the variance is the mean square of s - mu, taken from those registers (no
// cancellation for rows far from zero).  Statistics and sums are float32; the
// parameters' sums are float32 over at most 512 rows and 64-bit above.
// Bound by HBM bytes.  The backward's parameter sums stay in registers while
// a workgroup walks its rows; one partial per workgroup goes to the
// workspace, and a second launch adds the partials in a fixed order.
#include <algorithm>

#include "launch.hpp"
#include "row_ops.hpp"
#include "ssm.h"

namespace ssm {
namespace {

constexpr int block_of(int G) { return G > 256 ? G : 256; }

// Sum over the G lanes of a row; with G above a wavefront through LDS, one
// slot per wavefront, added in wavefront order.
template <int G, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*red)[K], int wv) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_reduce<(G < 64 ? G : 64), OpSum>(v[k]);
    if constexpr (G > 64) {
        constexpr int NW = G / 64;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[wv][k] = v[k];
        }
        __syncthreads();
        const int w0 = wv / NW * NW;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t = red[w0][k];
#pragma unroll
            for (int w = 1; w < NW; ++w) t += red[w0 + w][k];
            v[k] = t;
        }
    }
}

// A row of D values: `n` whole vectors dealt over its G lanes, NV to a lane
// (the fewest that hold them, so that only a lane's last can be past the end),
// and with EDGE D % VE > 0 values more, one to each of the first lanes.  Loads are
// not guarded but clamped to the row's last vector and masked afterwards: a
// load in a branch of its own is waited for there, and a lane's loads then
// follow each other one by one.
template <typename T, int NV, int G, bool EDGE, bool SHIFT = false>
struct RowOf {
    static constexpr int VE = kVec<T>, NR = NV > 0 ? NV : 1;
    int lane, n, tl;
    __device__ __forceinline__ RowOf(int lane_, int D) : lane(lane_), n(D / VE), tl(EDGE ? D % VE : 0) {}
    __device__ __forceinline__ int vec(int k) const { return lane + k * G; }
    __device__ __forceinline__ int place(int k) const { return k < NV - 1 ? vec(k) : min(vec(k), n - 1); }
    __device__ __forceinline__ bool has(int k) const { return k < NV - 1 || vec(k) < n; }
    __device__ __forceinline__ bool has_edge() const { return EDGE && lane < tl; }
    __device__ __forceinline__ int edge() const { return n * VE + (lane < tl ? lane : 0); }
    // Values as they came, the edge's too: its conversion here would wait for
    // the load (48756 x 2051 bfloat16 backward: 146 us, 165 with it).  SHIFT: a row that starts between two words is read a value
    // later, at word addresses (its edge makes sure that there is one), and the
    // vectors' first values on their own: 16-byte loads off a word's boundary
    // take long, which shows where few rows are in flight.
    struct Raw {
        u32x4 v[NR];
        T e, first[SHIFT ? NR : 1];
        uint32_t odd;
    };
    __device__ __forceinline__ void load(const T *row, Raw &f) const {
        f.odd = SHIFT ? (uint32_t)(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 1u : 0u;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            f.v[k] = *reinterpret_cast<const typename Unaligned16<T>::type *>(row + f.odd + place(k) * VE);
        if constexpr (SHIFT) {
            if (f.odd) {
#pragma unroll
                for (int k = 0; k < NV; ++k) f.first[k] = row[place(k) * VE];
            }
        }
        f.e = EDGE ? row[edge()] : T(0);
    }
    // the vectors, zeros past the end (and everywhere with !keep); the edge's value
    __device__ __forceinline__ float mask(Raw &f, bool keep) const {
        if constexpr (SHIFT) {
            if (f.odd) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const u32x4 q = f.v[k];
                    f.v[k] = u32x4{q[0] << 16 | (uint32_t)f.first[k], q[1] << 16 | q[0] >> 16, q[2] << 16 | q[1] >> 16,
                                   q[3] << 16 | q[2] >> 16};
                }
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (!(keep && has(k))) f.v[k] = splat4(0u);
        return keep && has_edge() ? to_f32(f.e) : 0.0f;
    }
    __device__ __forceinline__ void store(T *row, const float (&v)[NR][VE], float e) const {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (has(k)) *reinterpret_cast<typename Unaligned16<T>::type *>(row + vec(k) * VE) = pack(v[k], (const T *)nullptr);
        if (has_edge()) store_io(row + edge(), e);
    }
    // a float32 [D] parameter at this lane's values (`dflt` without one)
    __device__ __forceinline__ void param(const float *p, float dflt, float (&v)[NR][VE], float &e) const {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < VE; j += 4) {
                float q[4] = {dflt, dflt, dflt, dflt};
                if (p) {
                    const u32x4 r = *reinterpret_cast<const Unaligned16<float>::type *>(
                        p + place(k) * VE + j);
                    unpack(r, q, (const float *)nullptr);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[k][j + i] = q[i];
            }
        e = EDGE && p ? p[edge()] : dflt;
    }
};

template <typename T, int NV, int G, bool EDGE>
__global__ __launch_bounds__(block_of(G)) void norm_fwd_kernel(NormFwdArgs a) {
    constexpr int VE = kVec<T>, BLK = block_of(G), R = BLK / G, NR = NV > 0 ? NV : 1;
    __shared__ float red[2][BLK / 64][1];
    const int wv = threadIdx.x >> 6, D = (int)a.D;
    const RowOf<T, NV, G, EDGE> at(threadIdx.x % G, D);
    const int64_t row0 = (int64_t)blockIdx.x * R + (R > 1 ? threadIdx.x / G : 0);
    const bool act = row0 < a.T;               // a group past the last row works on that one and stores nothing
    const int64_t row = act ? row0 : a.T - 1;
    typename RowOf<T, NV, G, EDGE>::Raw x, r;
    float s[NR][VE];
    at.load(static_cast<const T *>(a.x) + row * a.x_stride, x);
    if (a.r) at.load(static_cast<const T *>(a.r) + row * a.r_stride, r);
    float es = at.mask(x, true);
#pragma unroll
    for (int k = 0; k < NV; ++k) unpack(x.v[k], s[k], (const T *)nullptr);
    if (a.r) {
        es += at.mask(r, true);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float q[VE];
            unpack(r.v[k], q, (const T *)nullptr);
#pragma unroll
            for (int i = 0; i < VE; ++i) s[k][i] += q[i];
        }
    }
    if (a.s != nullptr && act) at.store(static_cast<T *>(a.s) + row * a.s_stride, s, es);
    // the parameters arrive while the sums are taken
    float w[NR][VE], b[NR][VE], ew, eb;
    at.param(a.w, 1.0f, w, ew);
    at.param(a.b, 0.0f, b, eb);
    float m[1] = {es};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) m[0] += s[k][i];
    row_sums<G>(m, red[0], wv);
    const float mu = m[0] / (float)D;
    es = at.has_edge() ? es - mu : 0.0f;
    // squares are added as parts of their mean: 2^e, the largest power of two that
    // is at most 1 / D, changes no digit and keeps a wide row's sum of squares in
    // float32 as far as its mean square is
    const float part = __uint_as_float((uint32_t)(127 - (D > 1 ? 32 - __clz(D - 1) : 0)) << 23);
    float v[1] = {(es * part) * es};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            s[k][i] = at.has(k) ? s[k][i] - mu : 0.0f;
            v[0] = fmaf(s[k][i] * part, s[k][i], v[0]);
        }
    row_sums<G>(v, red[1], wv);
    const float rs = 1.0f / sqrtf(v[0] / ((float)D * part) + a.eps);
    if (!act) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) s[k][i] = fmaf(s[k][i] * rs, w[k][i], b[k][i]);
    es = fmaf(es * rs, ew, eb);
    at.store(static_cast<T *>(a.y) + row * a.y_stride, s, es);
    if (at.lane == 0) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = rs;
    }
}

// Rows are dealt round-robin to the workgroups' row groups.  AHEAD: the next
// row's loads are issued before this one's sums.
template <typename T, int NV, int G, bool EDGE>
__global__ __launch_bounds__(block_of(G)) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr int VE = kVec<T>, BLK = block_of(G), R = BLK / G, NR = NV > 0 ? NV : 1;
    // a CU holds one workgroup of 512 with 16 values to a lane: only this puts a
    // second row in flight there (19531 x 5120 bfloat16: 150 us, 175 without)
    constexpr bool AHEAD = G == 512 && sizeof(T) == 2;
    __shared__ float red[2][BLK / 64][2];
    const int wv = threadIdx.x >> 6, grp = R > 1 ? threadIdx.x / G : 0, D = (int)a.D;
    // 20000 x 4097 bfloat16: 142 us shifted, 174 not; 19996 x 5001: 193, 251; with
    // 128 lanes other rows hide the odd loads.  With 1024 lanes there are 128 registers,
    // and bfloat16 spills as it is (92 bytes a lane, 148 with an edge; float32 above
    // 8192 values 20 to 196): 11110 x 9000 bfloat16 306 us against 157 for its bytes,
    // 11109 x 9001 518, and 578 shifted
    using Row = RowOf<T, NV, G, EDGE, EDGE && sizeof(T) == 2 && (G == 256 || G == 512)>;
    const Row at(threadIdx.x % G, D);
    const float invD = 1.0f / (float)D;
    float w[NR][VE], dw[NR][VE], db[NR][VE], ew, edw = 0.0f, edb = 0.0f;
    at.param(a.w, 1.0f, w, ew);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) dw[k][i] = db[k][i] = 0.0f;
    struct In {
        typename Row::Raw x, dy, r;
        float mu, rs;
    } in{};
    auto fetch = [&](In &f, int64_t row) {
        row = min(row, a.T - 1);
        at.load(static_cast<const T *>(a.x) + row * a.x_stride, f.x);
        at.load(static_cast<const T *>(a.dy) + row * a.dy_stride, f.dy);
        if (a.dr) at.load(static_cast<const T *>(a.dr) + row * a.dr_stride, f.r);
        f.mu = a.mean[row];
        f.rs = a.rstd[row];
    };
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t row = (int64_t)blockIdx.x * R + grp;
    int par = 0;
    if constexpr (AHEAD) fetch(in, row);
    for (int64_t base = (int64_t)blockIdx.x * R; base < a.T; base += step, row += step, par ^= 1) {
        const bool act = row < a.T;            // a group past the last row loads that one and counts as zeros
        if constexpr (!AHEAD) fetch(in, row);
        typename Row::Raw r = in.r;
        const float ex = at.mask(in.x, act), ed = at.mask(in.dy, act);
        const float mu = act ? in.mu : 0.0f, rs = act ? in.rs : 0.0f;
        float xh[NR][VE], g[NR][VE];
        // past the row xh is 0: of a mean above 1e36 times rs it would be infinite, and 0 times that NaN
        float exh = (ex - mu) * (at.has_edge() ? rs : 0.0f), eg = ed * ew, c[2] = {eg, eg * exh};
        edw = fmaf(ed, exh, edw);
        edb += ed;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float d[VE];
            const float rk = at.has(k) ? rs : 0.0f;
            unpack(in.x.v[k], xh[k], (const T *)nullptr);
            unpack(in.dy.v[k], d, (const T *)nullptr);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                xh[k][i] = (xh[k][i] - mu) * rk;
                dw[k][i] = fmaf(d[i], xh[k][i], dw[k][i]);
                db[k][i] += d[i];
                g[k][i] = d[i] * w[k][i];
                c[0] += g[k][i];
                c[1] = fmaf(g[k][i], xh[k][i], c[1]);
            }
        }
        if constexpr (AHEAD) {
            if (base + step < a.T) fetch(in, row + step);
        }
        row_sums<G>(c, red[par], wv);
        if (a.dx != nullptr && act) {
            const float c0 = c[0] * invD, c1 = c[1] * invD;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < VE; ++i) g[k][i] = rs * (g[k][i] - c0 - xh[k][i] * c1);
            eg = rs * (eg - c0 - exh * c1);
            if (a.dr) {
                eg += at.mask(r, true);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    float q[VE];
                    unpack(r.v[k], q, (const T *)nullptr);
#pragma unroll
                    for (int i = 0; i < VE; ++i) g[k][i] += q[i];
                }
            }
            at.store(static_cast<T *>(a.dx) + row * a.dx_stride, g, eg);
        }
    }
    // this workgroup's partial sums: [2][D] (dw, then db), or the sums themselves
    // where it is the only one
    float *const ow = gridDim.x == 1 ? a.dw : a.ws + (int64_t)blockIdx.x * 2 * D;
    float *const ob = gridDim.x == 1 ? a.db : a.ws + (int64_t)blockIdx.x * 2 * D + D;
    if constexpr (R == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (at.has(k)) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    if (ow) ow[at.vec(k) * VE + i] = dw[k][i];
                    if (ob) ob[at.vec(k) * VE + i] = db[k][i];
                }
            }
        if (at.has_edge()) {
            if (ow) ow[at.edge()] = edw;
            if (ob) ob[at.edge()] = edb;
        }
    } else {
        constexpr int C = G * NV * VE + (EDGE ? VE : 0);     // columns a row group holds
        __shared__ float acc[R][C];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h) __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (at.has(k)) acc[grp][at.vec(k) * VE + i] = h ? db[k][i] : dw[k][i];
            if (at.has_edge()) acc[grp][at.edge()] = h ? edb : edw;
            __syncthreads();
            float *const out = h ? ob : ow;
            for (int c = threadIdx.x; out != nullptr && c < D; c += BLK) {
                float t = acc[0][c];
#pragma unroll
                for (int q = 1; q < R; ++q) t += acc[q][c];
                out[c] = t;
            }
        }
    }
}

// dw, db: the partials of every workgroup, added in 64 bits (there are as many as
// the rows make).  32 columns x 32 strips of partials per workgroup (128-byte
// reads); strips added in order.
__global__ __launch_bounds__(1024) void norm_bwd_reduce(const float *ws, int64_t P, int64_t D, float *dw, float *db) {
    __shared__ double part[32][33];
    const int cl = threadIdx.x & 31, st = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + cl;
    double t = 0.0;
    if (c < 2 * D) {
#pragma unroll 8
        for (int64_t p = st; p < P; p += 32) t += (double)ws[p * 2 * D + c];
    }
    part[st][cl] = t;
    __syncthreads();
    if (st == 0 && c < 2 * D) {
#pragma unroll
        for (int k = 1; k < 32; ++k) t += part[k][cl];
        if (c < D) {
            if (dw) dw[c] = (float)t;
        } else if (db) {
            db[c - D] = (float)t;
        }
    }
}

// Lanes of a row: the fewest (from 16 on) that hold its whole vectors in at
// most `most` each.
int row_lanes(int64_t n, int most) {
    int G = 16;
    while (G < 1024 && (int64_t)G * most < n) G *= 2;
    return G;
}

// Vectors of a lane at most.  Forward, 16384 x 384: float32 18.8 us with 2,
// 20.9 with 4, 19.8 with 1; bfloat16 10.2 with 4, 10.6 with 2, and 49.4
// against 50.4 at 16384 x 2048.  Backward: float32 16384 x 384 20.5 us with 2,
// 21.7 with 4; bfloat16 20011 x 2048 62.5 with 2, 64.2 with 4, 65.9 with 1.
template <typename T> constexpr int kFwdVecs = sizeof(T) == 4 ? 2 : 4;
constexpr int kBwdVecs = 2;

// Workgroups of the backward: two per CU, one where a row takes 512 lanes or
// more.  In bfloat16 a CU holds one of those (162 and 182 registers; 19531 x 5120:
// 151 us, 167 with two), in float32 two (88 and 100), but one with half the
// partial sums is the faster from 4096 values on: with dresidual 16384 x 4096 190 us
// against 206, 12000 x 5120 179 and 193, 8192 x 8192 205 and 212, 4096 x 16384 315
// and 342 (20000 x 2560 165 and 165, without dresidual 139 and 118);
// fewer where the rows run out; one alone for rows that it takes in two goes (a
// third costs what the launch of the sums does); more where a row group would add
// more than kChain rows to its float32 parameter sums, whose error grows with them (as
// many for each CU: 300001 x 4104 bfloat16 1519 us with 768 workgroups, 1872 with
// the 586 that would do, 1481 with 256 that add 1172 rows each).
constexpr int64_t kChain = 512;
int64_t bwd_blocks(int64_t T, int64_t D, int bf16) {
    const int G = row_lanes(D / (bf16 ? kVec<bf16_t> : kVec<float>), kBwdVecs);
    const int64_t R = block_of(G) / G;
    const int64_t resident = G >= 512 ? 256 : 512, most = resident * R * kChain;
    return T <= 2 * R ? 1 : std::min((T + R - 1) / R, resident * ((T + most - 1) / most));
}

struct Fwd {
    static constexpr int kind = 0;
};
struct Bwd {
    static constexpr int kind = 1;
};
template <typename K, typename T, int NV, int G, bool EDGE, typename A>
void go(const A &a, hipStream_t s) {
    if constexpr (K::kind == 0) {
        // a launch has fewer than 2^32 threads
        constexpr int64_t R = block_of(G) / G, kRows = ((int64_t)1 << 31) / block_of(G) * R;
        for (int64_t t = 0; t < a.T; t += kRows) {
            A b = a;
            b.T = std::min(kRows, a.T - t);
            b.x = static_cast<const T *>(a.x) + t * a.x_stride;
            b.r = a.r ? static_cast<const T *>(a.r) + t * a.r_stride : nullptr;
            b.s = a.s ? static_cast<T *>(a.s) + t * a.s_stride : nullptr;
            b.y = static_cast<T *>(a.y) + t * a.y_stride;
            b.mean = a.mean ? a.mean + t : nullptr;
            b.rstd = a.rstd ? a.rstd + t : nullptr;
            hipLaunchKernelGGL((norm_fwd_kernel<T, NV, G, EDGE>), dim3((unsigned)((b.T + R - 1) / R)),
                               dim3(block_of(G)), 0, s, b);
        }
    } else {
        hipLaunchKernelGGL((norm_bwd_kernel<T, NV, G, EDGE>), dim3((unsigned)bwd_blocks(a.T, a.D, a.bf16)),
                           dim3(block_of(G)), 0, s, a);
    }
}
// The variant with exactly this many vectors to a lane: above 16 lanes more
// than half of MOST.
template <typename K, typename T, int G, int NV, int MOST, typename A>
void pick_vecs(const A &a, int nv, hipStream_t s) {
    if (nv == NV) {
        if constexpr (NV > 0) {
            if (a.D % kVec<T> == 0) return go<K, T, NV, G, false>(a, s);
        }
        go<K, T, NV, G, true>(a, s);
    } else if constexpr (NV < MOST)
        pick_vecs<K, T, G, NV + 1, MOST>(a, nv, s);
}
template <typename K, typename T, int MOST, typename A>
hipError_t launch_rows(const A &a, hipStream_t s) {
    const int64_t n = a.D / kVec<T>;
    const int G = row_lanes(n, MOST), nv = (int)((n + G - 1) / G);
    constexpr int LEAST = MOST / 2 + 1;
    switch (G) {
        case 16: pick_vecs<K, T, 16, 0, MOST>(a, nv, s); break;
        case 32: pick_vecs<K, T, 32, LEAST, MOST>(a, nv, s); break;
        case 64: pick_vecs<K, T, 64, LEAST, MOST>(a, nv, s); break;
        case 128: pick_vecs<K, T, 128, LEAST, MOST>(a, nv, s); break;
        case 256: pick_vecs<K, T, 256, LEAST, MOST>(a, nv, s); break;
        case 512: pick_vecs<K, T, 512, LEAST, MOST>(a, nv, s); break;
        default: pick_vecs<K, T, 1024, LEAST, std::max(MOST, SSM_MAX_NORM_DIM / kVec<T> / 1024)>(a, nv, s); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdArgs &a, hipStream_t s) {
    if (a.T == 0) return hipSuccess;
    return a.bf16 ? launch_rows<Fwd, bf16_t, kFwdVecs<bf16_t>>(a, s) : launch_rows<Fwd, float, kFwdVecs<float>>(a, s);
}

size_t norm_bwd_workspace_bytes(int64_t T, int64_t D, int bf16) {
    return ws_align((size_t)(std::max<int64_t>(1, bwd_blocks(T, D, bf16)) * 2 * D) * sizeof(float));
}

hipError_t launch_norm_bwd(const NormBwdArgs &a, hipStream_t s) {
    const int64_t P = a.T > 0 ? bwd_blocks(a.T, a.D, a.bf16) : 0;
    if (P > 0) {
        const hipError_t e = a.bf16 ? launch_rows<Bwd, bf16_t, kBwdVecs>(a, s) : launch_rows<Bwd, float, kBwdVecs>(a, s);
        if (e != hipSuccess) return e;
    }
    if (P == 1 || (a.dw == nullptr && a.db == nullptr)) return hipSuccess;
    hipLaunchKernelGGL(norm_bwd_reduce, dim3((unsigned)((2 * a.D + 31) / 32)), dim3(1024), 0, s, a.ws, P, a.D, a.dw,
                       a.db);
    return hipGetLastError();
}

}  // namespace ssm
