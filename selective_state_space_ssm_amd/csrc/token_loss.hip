// token_loss.hip -- log-probabilities of chosen tokens and the clipped policy
// loss, from rows of V logits, with their gradients.
//
// With m = max_j z_j and l = log sum_j exp(z_j - m), a token a of a row has
//   logp = z_a - m - l,   d logp / d z_j = [j = a] - exp(z_j - m - l).
// The policy loss of a counted token with weight w, advantage A, ratio
// r = exp(logp - old) and gap d = ref - logp is
//   w (-min(r A, clip(r, lo, hi) A) + beta (exp(d) - 1 - d)),
// so dloss/dlogp = w (-A r [not clipped] - beta (exp(d) - 1)).
//
// exp is 2^x of the float32 difference z - m (never of z itself: a row of the
// type's lowest values is a uniform row); sums over a lane's share and over
// 16 lanes are float32, which leaves errors of up to 3e-7 in log p, to either
// side (6e-8 to 9e-8 in the mean square over rows of 60 to 70001 logits).
// Everything after them is 64-bit and adds nothing to that: whether a ratio is
// clipped is decided next to a border.  Bound by HBM bytes: the forward reads
// the logits once (a running maximum and sum per lane), the policy loss keeps
// a row in registers between its maximum, its sum and its gradient, so the
// logits are read once and the gradient is written once.
#include <algorithm>

#include "launch.hpp"
#include "row_ops.hpp"

namespace ssm {
namespace {

constexpr int block_of(int G) { return G > 256 ? G : 256; }
constexpr float kNegInf = -__builtin_huge_valf();

// -inf in every value of a raw vector
template <typename T> constexpr uint32_t kNegInfRaw = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;

__device__ __forceinline__ float safe_max(float m) { return m == kNegInf ? 0.0f : m; }

// e^x of the sums: 2^(x log2 e) with log2 e in two floats and one rounding.  x times
// the first alone makes every term 1.3e-8 |x| too large, which no averaging takes
// out of log sum (4e-8 at 4096 logits of deviation 2.5); the hardware's 2^x is off
// by -3e-9 on the average.  One instruction more: log-probabilities of 8192 x 50001
// bfloat16 137.5 us (136.4 without), the policy loss at 16384 x 2048 36.1 (34.8).  The
// gradients' exponentials are not summed and go without: 1.3e-8 |x| of e^x each.
constexpr float kLog2eLow = 1.92596299e-8f;
__device__ __forceinline__ float exp_term(float x) { return hw_exp2(fmaf(x, kLog2e, x * kLog2eLow)); }

// e^x and e^x - 1 in 64 bits, to about 1e-11: x = k ln 2 + f with |f| <= ln 2 / 2,
// e^f - 1 by its Taylor series to f^10 (the next term is below 3e-13 of e^f),
// then 2^k (e^f - 1) + (2^k - 1).  The 64-bit library functions' constants
// stayed in registers through the row loop: 133 of them against 72 (V 4096,
// float32), and three wavefronts on a SIMD instead of seven.
struct Exp {
    double e, em1;
};
__device__ __forceinline__ Exp exp_f64(double x) {
    const double c = fmin(fmax(x, -1000.0), 1000.0);          // e^x is 0 or infinite beyond
    const double k = rint(c * 1.4426950408889634);
    // ln 2 in two parts, the first of 32 bits: its product with k is exact
    const double f = fma(k, 4.2009150726810846e-11, fma(k, -0.6931471806019545, c));
    double p = 1.0 / 3628800.0;
    p = fma(p, f, 1.0 / 362880.0);
    p = fma(p, f, 1.0 / 40320.0);
    p = fma(p, f, 1.0 / 5040.0);
    p = fma(p, f, 1.0 / 720.0);
    p = fma(p, f, 1.0 / 120.0);
    p = fma(p, f, 1.0 / 24.0);
    p = fma(p, f, 1.0 / 6.0);
    p = fma(p, f, 0.5);
    p = fma(p * f, f, f);
    const int n = (int)k;
    Exp r;
    r.e = x != x ? x : ldexp(1.0 + p, n);
    r.em1 = fabs(k) > 60.0 || x != x ? r.e - 1.0 : ldexp(p, n) + (ldexp(1.0, n) - 1.0);
    return r;
}

// log(s) in 64 bits for s >= 1 (NaN for NaN): the hardware's log2 corrected by
// log(1 + d), d = s e^-y - 1 of about 1e-7.
__device__ __forceinline__ double log_f64(double s) {
    const double y = (double)hw_log2((float)s) * 0.69314718055994530942;
    const double d = fma(s, exp_f64(-y).e, -1.0);
    return y + (d - 0.5 * d * d);
}

// Joins the lanes' (m, s) -- maximum and sum of exp(z - safe_max(m)) -- over
// the G lanes of a row: m becomes the row's maximum, and the sum is returned
// in 64 bits.  With G above a wavefront through LDS, one barrier (`red` must
// not be written again before every wavefront has passed another barrier, or
// be another buffer).
template <int G>
__device__ __forceinline__ double join(float &m, float s, float *red_m, double *red_s, int wv) {
    static_assert(G >= 64, "a row has whole wavefronts");
    const float mw = lanes_reduce<64, OpMax>(m);
    if (m != kNegInf) s *= exp_term(m - mw);        // a lane of -inf keeps its 0 (or NaN)
    s = lanes_reduce<16, OpSum>(s);
    double t = ((double)lane_of(s, 0) + (double)lane_of(s, 16)) + ((double)lane_of(s, 32) + (double)lane_of(s, 48));
    m = mw;
    if constexpr (G > 64) {
        constexpr int NW = G / 64;
        static_assert(NW == 4 || NW == 8 || NW == 16, "wavefronts of a row");
        if ((threadIdx.x & 63) == 0) {
            red_m[wv] = mw;
            red_s[wv] = t;
        }
        __syncthreads();
        // every wavefront joins the others' results, a lane for each
        const int w = threadIdx.x & (NW - 1);
        const float q = red_m[w];
        t = red_s[w];
        m = fmaxf(q, dpp_f<kDppQuadSwap1>(q));
        m = fmaxf(m, dpp_f<kDppQuadSwap2>(m));
        if constexpr (NW >= 8) m = fmaxf(m, dpp_f<kDppRowHalfMirror>(m));
        if constexpr (NW >= 16) m = fmaxf(m, dpp_f<kDppRowMirror>(m));
        t *= (double)(q == kNegInf ? 1.0f : exp_term(q - m));
        t += dpp_f64<kDppQuadSwap1>(t);
        t += dpp_f64<kDppQuadSwap2>(t);
        if constexpr (NW >= 8) t += dpp_f64<kDppRowHalfMirror>(t);
        if constexpr (NW >= 16) t += dpp_f64<kDppRowMirror>(t);
    }
    return t;
}

// A row of V values is a head, whole vectors and a tail; the row's first lanes
// take a value of the head or the tail each, so no vector needs a guard inside.
template <typename T>
__device__ __forceinline__ u32x4 ld16(const T *row, int vec) {
    return *reinterpret_cast<const typename Unaligned16<T>::type *>(reinterpret_cast<const char *>(row) +
                                                                    (uint32_t)vec * 16u);
}
// `vec`, or where the row has no such vector the last one it has: the load
// itself is not guarded, because a load in a branch of its own is waited for
// there, one after the other (the caller masks the value).
template <typename T>
__device__ __forceinline__ u32x4 ld16_clamped(const T *row, int vec, int nf) {
    return ld16(row, min(vec, nf - 1));
}
template <typename T>
__device__ __forceinline__ void st16(T *row, int vec, const u32x4 &v) {
    *reinterpret_cast<typename Unaligned16<T>::type *>(reinterpret_cast<char *>(row) + (uint32_t)vec * 16u) = v;
}
template <typename T>
struct Cut {
    int hd, nf, tl;                            // values of the head, whole vectors, values of the tail
    __device__ __forceinline__ explicit Cut(int V) : hd(0), nf(V / kVec<T>), tl(V % kVec<T>) {}
    // cut so that the vectors start on 16 bytes: rows of an odd length read
    // from where they begin took 172 us against 144 (8192 x 50001 bf16)
    __device__ __forceinline__ Cut(const T *row, int V)
        : hd(min(V, (int)((0u - (uint32_t)(reinterpret_cast<uintptr_t>(row) / sizeof(T))) & (kVec<T> - 1)))),
          nf((V - hd) / kVec<T>), tl((V - hd) % kVec<T>) {}
    // the head's and the tail's value this lane has (-1: none)
    __device__ __forceinline__ int edge(int lane) const {
        return lane < hd ? lane : (lane >= kVec<T> && lane < kVec<T> + tl ? hd + nf * kVec<T> + lane - kVec<T> : -1);
    }
    __device__ __forceinline__ float edge_value(const T *row, int lane) const {
        const int e = edge(lane);
        return e >= 0 ? to_f32(row[e]) : kNegInf;
    }
};

// One pass over a row in memory: the lane's running maximum and sum, U
// vectors between two rescalings.
template <typename T, int G, int U, bool WHOLE>
__device__ __forceinline__ void scan_block(const T *z, int nf, int i0, float &m, float &s) {
    constexpr int VE = kVec<T>;
    u32x4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = WHOLE ? ld16(z, i0 + u * G) : ld16_clamped(z, i0 + u * G, nf);
    if constexpr (!WHOLE) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * G >= nf) raw[u] = splat4(kNegInfRaw<T>);
    }
    float v[U][VE], cm = kNegInf;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        unpack(raw[u], v[u], (const T *)nullptr);
#pragma unroll
        for (int i = 0; i < VE; ++i) cm = fmaxf(cm, v[u][i]);
    }
    const float mn = fmaxf(m, cm), ref = safe_max(mn);
    float t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < VE; ++i) t[i & 1] += exp_term(v[u][i] - ref);
    s = (m == kNegInf ? s : s * exp_term(m - ref)) + (t[0] + t[1]);
    m = mn;
}
template <typename T, int G, int U>
__device__ __forceinline__ void scan_row(const T *z, const Cut<T> &c, int lane, float &m, float &s) {
    m = c.edge_value(z, lane);
    s = m == m ? (m == kNegInf ? 0.0f : 1.0f) : m;
    z += c.hd;
    int b = 0;
    for (; b + G * U <= c.nf; b += G * U) scan_block<T, G, U, true>(z, c.nf, b + lane, m, s);
    if (b < c.nf) scan_block<T, G, U, false>(z, c.nf, b + lane, m, s);
}

template <typename T, int G>
__global__ __launch_bounds__(block_of(G)) void logp_fwd_kernel(LogpArgs a) {
    constexpr int BLK = block_of(G), R = BLK / G;
    __shared__ float red_m[BLK / 64];
    __shared__ double red_s[BLK / 64];
    const int lane = threadIdx.x % G, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = (int64_t)blockIdx.x * R + (R == 1 ? 0 : wv);
    if (row >= a.T) return;                    // whole wavefronts; with barriers R is 1
    const int V = (int)a.V;
    const int32_t t = a.tgt[row];
    if (t < 0) {                               // no target: the row is not read
        if (lane == 0) {
            a.logp[row] = 0.0f;
            if (a.stats) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
        }
        return;
    }
    const T *z = static_cast<const T *>(a.z) + row * a.z_stride;
    const float za = t < V ? to_f32(z[t]) : __builtin_nanf("");
    float m, s;
    scan_row<T, G, 4>(z, Cut<T>(z, V), lane, m, s);
    const double sum = join<G>(m, s, red_m, red_s, wv);
    if (lane == 0) {
        const double l = log_f64(sum);
        a.logp[row] = (float)(((double)za - (double)m) - l);
        if (a.stats) {
            a.stats[2 * row] = m;
            a.stats[2 * row + 1] = (float)l;
        }
    }
}

// dz of one chunk of a row: G lanes, U vectors each; the row's last chunk has
// its tail.
template <typename T, int G, int U>
__global__ __launch_bounds__(256) void logp_bwd_kernel(LogpArgs a, int chunks) {
    constexpr int VE = kVec<T>, R = 256 / G;
    const int lane = threadIdx.x % G, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = (int64_t)blockIdx.x * R + (R == 1 ? 0 : wv);
    const int64_t row = R == 1 ? id / chunks : id;            // with R > 1 a row is one chunk
    if (row >= a.T) return;
    const int V = (int)a.V, chunk = R == 1 ? (int)(id - row * chunks) : 0;
    const Cut<T> c(V);
    const int i0 = chunk * (G * U) + lane;
    const int tail = chunk == chunks - 1 ? c.edge(lane) : -1;
    const int32_t t = a.tgt[row];
    const float d = t < 0 ? 0.0f : a.dlogp[row];
    T *dz = static_cast<T *>(a.dz) + row * a.dz_stride;
    if (d == 0.0f) {                           // the row's logits are not read
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * G < c.nf) st16(dz, i0 + u * G, splat4(0u));
        if (tail >= 0) store_io(dz + tail, 0.0f);
        return;
    }
    const T *z = static_cast<const T *>(a.z) + row * a.z_stride;
    u32x4 raw[U];
    if (c.nf > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = ld16_clamped(z, i0 + u * G, c.nf);
    }
    const float zt = tail >= 0 ? to_f32(z[tail]) : 0.0f;
    const float m = a.stats_in[2 * row], l = a.stats_in[2 * row + 1], l2 = l * kLog2e;
    const float nd = t < V ? -d : __builtin_nanf("");
    // at the target d (1 - p), without the cancellation next to p = 1
    auto at_target = [&](float v) { return -d * expm1f((v - m) - l); };
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int vec = i0 + u * G;
        if (vec >= c.nf) break;
        float v[VE], gt = 0.0f;
        unpack(raw[u], v, (const T *)nullptr);
        const int ti = t - vec * VE;
        if ((unsigned)ti < (unsigned)VE) {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (i == ti) gt = at_target(v[i]);
        }
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            v[i] = nd * hw_exp2(fmaf(v[i] - m, kLog2e, -l2));
            if (i == ti) v[i] = gt;
        }
        st16(dz, vec, pack(v, (const T *)nullptr));
    }
    if (tail >= 0) store_io(dz + tail, tail == t ? at_target(zt) : nd * hw_exp2(fmaf(zt - m, kLog2e, -l2)));
}

// ------------------------------------------------------------ policy loss
// Workspace: [kWeightParts] sums of weights, then [blocks][4] sums of the
// loss, its policy term, the KL term and the clipped tokens' weights.
constexpr int kWeightParts = 64;
constexpr int kOwnWeights = 512;

__device__ __forceinline__ float token_weight(const PolicyArgs &a, int64_t row) {
    const float w = a.wt ? a.wt[row] : 1.0f;
    return a.tgt[row] < 0 ? 0.0f : w;
}

__global__ __launch_bounds__(256) void policy_weights_kernel(PolicyArgs a) {
    __shared__ double part[4];
    double t = 0.0;
#pragma unroll 8
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.T; i += (int64_t)gridDim.x * 256)
        t += (double)token_weight(a, i);
    t = wave_sum_f64(t);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) a.ws[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// 1 / sum of the counted tokens' weights (0 when there is nothing to divide
// by, 1 for a sum over tokens); all 64 lanes of the wavefront must be active.
// `parts` 0: summed here from the weights themselves.
__device__ __forceinline__ double load_weights(const PolicyArgs &a, int parts) {
    const int l = threadIdx.x & 63;
    double w = 0.0;
    if (!a.mean) return w;
    if (parts > 0) return l < parts ? a.ws[l] : 0.0;
#pragma unroll 4
    for (int i = l; i < (int)a.T; i += 64) w += (double)token_weight(a, i);
    return w;
}
__device__ __forceinline__ double inv_weights(const PolicyArgs &a, double part) {
    if (!a.mean) return 1.0;
    const double w = wave_sum_f64(part);
    return w == 0.0 ? 0.0 : 1.0 / w;
}

// A token's inputs, and what it adds to the loss.
struct Token {
    int t;                                     // target
    float w, adv, old_logp, ref_logp;
};
__device__ __forceinline__ Token load_token(const PolicyArgs &a, int64_t row) {
    row = min(row, a.T - 1);                   // past the last row: loaded, not used
    Token o;
    o.t = a.tgt[row];
    o.w = a.wt ? a.wt[row] : 1.0f;
    o.adv = a.adv[row];
    o.old_logp = a.old_logp ? a.old_logp[row] : 0.0f;
    o.ref_logp = a.ref_logp ? a.ref_logp[row] : 0.0f;
    return o;
}
struct Terms {
    double loss, pg, kl, clip, grad, pm1;      // grad: dloss/dlogp; pm1: p - 1
};
__device__ __forceinline__ Terms token_terms(const PolicyArgs &a, const Token &k, double logp) {
    // r, e^d - 1 and p - 1 by one evaluation, a lane each
    const int l = threadIdx.x & 63;
    const double x0 = a.old_logp ? logp - (double)k.old_logp : (logp == logp ? 0.0 : logp);
    const double d = a.ref_logp ? (double)k.ref_logp - logp : 0.0;
    const Exp v = exp_f64(l == 0 ? x0 : (l == 1 ? d : logp));
    const double r = lane_f64(v.e, 0), e = lane_f64(v.em1, 1);
    const double adv = (double)k.adv;
    Terms o;
    o.pm1 = lane_f64(v.em1, 2);
    const bool clip = adv > 0.0 ? r > a.hi : (adv < 0.0 && r < a.lo);
    const double held = (adv > 0.0 ? a.hi : a.lo) * adv;
    o.pg = clip ? -held : -(r * adv);
    o.clip = clip ? 1.0 : 0.0;
    o.grad = clip ? 0.0 : -(r * adv);
    o.kl = e - d;
    o.loss = o.pg;
    if (a.beta != 0.0) {
        o.loss += a.beta * o.kl;
        o.grad -= a.beta * e;
    }
    return o;
}

template <typename T, int G>
__device__ __forceinline__ void zero_row(T *dz, const Cut<T> &c, int lane) {
    for (int i = lane; i < c.nf; i += G) st16(dz + c.hd, i, splat4(0u));
    if (c.edge(lane) >= 0) store_io(dz + c.edge(lane), 0.0f);
}

// One vector of dz = k * exp(z - ref), the target's value (place ti of the
// vector, if it has one) replaced by gt.
template <typename T>
__device__ __forceinline__ u32x4 grad_vec(const u32x4 &raw, float ref, float k, int ti, float gt) {
    constexpr int VE = kVec<T>;
    float v[VE];
    unpack(raw, v, (const T *)nullptr);
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = k * hw_exp2((v[i] - ref) * kLog2e);
    if ((unsigned)ti < (unsigned)VE) {
#pragma unroll
        for (int i = 0; i < VE; ++i)
            if (i == ti) v[i] = gt;
    }
    return pack(v, (const T *)nullptr);
}

// Keeps the raw vectors as they are between two passes over them: otherwise
// the compiler carries the unpacked values and their exponentials along (a
// row of 8 bf16 vectors then took 207 registers or spilled).
template <int N>
__device__ __forceinline__ void hold(u32x4 (&raw)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) asm volatile("" : "+v"(raw[k]));
}

// G lanes a row.  NV > 0: the row in NV vectors a lane, read once; NV = 0:
// any length, read again for the gradient.
template <typename T, int NV, int G>
__global__ __launch_bounds__(block_of(G)) void policy_kernel(PolicyArgs a, int parts) {
    constexpr int VE = kVec<T>, BLK = block_of(G), R = BLK / G;
    __shared__ float red_m[2][BLK / 64];
    __shared__ double red_s[2][BLK / 64];
    __shared__ double sums[R][4];
    int lane = threadIdx.x % G;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = R == 1 ? 0 : wv;
    const int V = (int)a.V;
    const double wpart = load_weights(a, parts);
    double inv = -1.0, acc[4] = {0.0, 0.0, 0.0, 0.0};
    int64_t row = (int64_t)blockIdx.x * R + grp;
    const int64_t step = (int64_t)gridDim.x * R;
    Token next = load_token(a, row);
    for (int par = 0; row < a.T; row += step) {
        asm volatile("" : "+v"(lane));         // what follows from it is cheaper made anew than kept
        Token tok = next;
        if (tok.t < 0) tok.w = 0.0f;
        next = load_token(a, row + step);
        T *dz = a.dz ? static_cast<T *>(a.dz) + row * a.dz_stride : nullptr;
        if (tok.w == 0.0f) {                   // left out, the same for every lane: nothing of it is read
            if (dz) zero_row<T, G>(dz, Cut<T>(dz, V), lane);
            if (a.logp && lane == 0) a.logp[row] = 0.0f;
        } else {
            const T *z = static_cast<const T *>(a.z) + row * a.z_stride;
            const Cut<T> c(z, V);
            const float target = tok.t < V ? to_f32(z[tok.t]) : __builtin_nanf("");
            u32x4 raw[NV > 0 ? NV : 1];
            float edge = 0.0f, m = kNegInf, s = 0.0f;
            if constexpr (NV > 0) {
                // NV is the fewest vectors that hold a row of V values, so only the
                // last can be past its end
#pragma unroll
                for (int q = 0; q < NV - 1; ++q) raw[q] = ld16(z + c.hd + q * G * VE, lane);
                raw[NV - 1] = ld16_clamped(z + c.hd, lane + (NV - 1) * G, c.nf);
                if (inv < 0.0) inv = inv_weights(a, wpart);      // while the row is on its way
                if (lane >= c.nf - (NV - 1) * G) raw[NV - 1] = splat4(kNegInfRaw<T>);
                m = edge = c.edge_value(z, lane);
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    float v[VE];
                    unpack(raw[q], v, (const T *)nullptr);
#pragma unroll
                    for (int i = 0; i < VE; ++i) m = fmaxf(m, v[i]);
                }
                hold(raw);
                const float ref = safe_max(m);
                s = exp_term(edge - ref);
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    float v[VE];
                    unpack(raw[q], v, (const T *)nullptr);
                    float u = 0.0f;
#pragma unroll
                    for (int i = 0; i < VE; ++i) u += exp_term(v[i] - ref);
                    s += u;
                }
            } else {
                if (inv < 0.0) inv = inv_weights(a, wpart);
                scan_row<T, G, 4>(z, c, lane, m, s);
            }
            const double sum = join<G>(m, s, red_m[par], red_s[par], wv);
            par ^= 1;
            const double logp = ((double)target - (double)m) - log_f64(sum);
            const Terms o = token_terms(a, tok, logp);
            if (lane == 0) {
                const double dw = (double)tok.w;
                acc[0] += dw * o.loss;
                acc[1] += dw * o.pg;
                acc[2] += dw * o.kl;
                acc[3] += dw * o.clip;
                if (a.logp) a.logp[row] = (float)logp;
            }
            if (dz) {
                const double g = o.grad * (double)tok.w * inv * a.gscale;
                const float gt = (float)(-g * o.pm1), k = (float)-g / (float)sum, ref = safe_max(m);
                if constexpr (NV > 0) {
                    hold(raw);
#pragma unroll
                    for (int q = 0; q < NV; ++q)
                        if (q < NV - 1 || lane < c.nf - q * G)
                            st16(dz + c.hd + q * G * VE, lane,
                                 grad_vec<T>(raw[q], ref, k, tok.t - c.hd - q * G * VE - lane * VE, gt));
                } else {
                    for (int i = lane; i < c.nf; i += G)
                        st16(dz + c.hd, i, grad_vec<T>(ld16(z + c.hd, i), ref, k, tok.t - c.hd - i * VE, gt));
                }
                const int i = c.edge(lane);
                if (i >= 0) {
                    const float v = NV > 0 ? edge : c.edge_value(z, lane);
                    store_io(dz + i, i == tok.t ? gt : k * hw_exp2((v - ref) * kLog2e));
                }
            }
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[grp][q] = acc[q];
    }
    __syncthreads();
    // a workgroup that is the only one has the loss; of several each leaves a sum
    const bool alone = gridDim.x == 1;
    if (alone) inv = inv_weights(a, wpart);
    if (threadIdx.x < 4) {
        double t = sums[0][threadIdx.x];
#pragma unroll
        for (int g = 1; g < R; ++g) t += sums[g][threadIdx.x];
        if (alone)
            a.loss[threadIdx.x] = (float)(t * inv);
        else
            a.ws[kWeightParts + (int64_t)blockIdx.x * 4 + threadIdx.x] = t;
    }
}

// A launch of its own: letting the workgroup that finishes last add the sums
// needs a release by each, which writes its XCD's L2 back (about 0.1 us a
// workgroup: 283 us against 115 with 2048 of them).
__global__ __launch_bounds__(1024) void policy_finish_kernel(PolicyArgs a, int parts, int blocks) {
    __shared__ double part[16][4];
    const int q = threadIdx.x & 3;             // which of the four sums
    const double wpart = load_weights(a, parts);
    double t = 0.0;
#pragma unroll 4
    for (int b = threadIdx.x >> 2; b < blocks; b += 256) t += a.ws[kWeightParts + 4 * b + q];
    const double inv = inv_weights(a, wpart);
#pragma unroll
    for (int o = 4; o < 64; o <<= 1) t += __shfl_xor(t, o, 64);
    if ((threadIdx.x & 63) < 4) part[threadIdx.x >> 6][q] = t;
    __syncthreads();
    if (threadIdx.x < 4) {
        double u = part[0][q];
#pragma unroll
        for (int w = 1; w < 16; ++w) u += part[w][q];
        a.loss[q] = (float)(u * inv);
    }
}

// Lanes of a row, and how many vectors of it each holds (0: it is read twice).
// A vector's place moves with the row's alignment: V / ve of them at most, one
// fewer at least.  A wavefront to a row up to 512 vectors (16384 x 4096
// bfloat16: 52 us, 66 with a workgroup of 256 each; 16384 x 2048: 32, 53); 256
// lanes up to 2048 (16384 x 4096 float32: 103 us, 110 with a wavefront, 122
// with 512); 512 beyond (4096 x 50001 bfloat16: 151 us with the small launches,
// 188 with 1024).
struct RowPlan {
    int G, NV;
};
RowPlan plan_row(int64_t V, int ve) {
    const int64_t n = V / ve;                  // whole vectors
    if (n < 2) return RowPlan{64, 0};          // (a row may have none)
    const int G = n <= 64 * 8 ? 64 : n <= 256 * 8 ? 256 : n <= 512 * 16 ? 512 : 1024;
    const int64_t NV = (n + G - 1) / G;
    return NV <= 16 ? RowPlan{G, (int)NV} : RowPlan{1024, 0};
}

// A workgroup for each row (G = 64: four rows), up to what the last launch
// adds in passing; one alone, without that launch, for one row or two short ones
// to a wavefront (11.0 us a call, 13.2 with it; two rows of 50001 one after the
// other 16.6, side by side 13.9).
int64_t policy_blocks(int64_t T, int64_t V, int bf16) {
    const RowPlan p = plan_row(V, bf16 ? kVec<bf16_t> : kVec<float>);
    const int64_t R = block_of(p.G) / p.G;
    return T > 0 && T <= (R > 1 ? 2 * R : 1) ? 1 : std::min<int64_t>(8192, (T + R - 1) / R);
}

template <typename T, int G, int NV, int LAST>
void go_policy(int nv, const PolicyArgs &a, int parts, int64_t blocks, hipStream_t s) {
    if (nv == NV)
        hipLaunchKernelGGL((policy_kernel<T, NV, G>), dim3((unsigned)blocks), dim3(block_of(G)), 0, s, a, parts);
    else if constexpr (NV < LAST)
        go_policy<T, G, NV + 1, LAST>(nv, a, parts, blocks, s);
}

template <typename T>
void launch_policy_t(const PolicyArgs &a, int parts, int64_t blocks, hipStream_t s) {
    const RowPlan p = plan_row(a.V, kVec<T>);
    switch (p.G) {
        case 64: return go_policy<T, 64, 0, 8>(p.NV, a, parts, blocks, s);
        case 256: return go_policy<T, 256, 3, 8>(p.NV, a, parts, blocks, s);
        case 512: return go_policy<T, 512, 5, 16>(p.NV, a, parts, blocks, s);
        default:
            if (p.NV == 0) return go_policy<T, 1024, 0, 0>(0, a, parts, blocks, s);
            return go_policy<T, 1024, 9, 16>(p.NV, a, parts, blocks, s);
    }
}

// Lanes of a row: a wavefront, four rows to a workgroup, where the rows are
// short (16384 x 4096 bfloat16: 23 us, 35 with a workgroup each, which is what
// starting 16384 workgroups takes); 512 where they are long (8192 x 50001
// bfloat16: 137 us, 144 with 256; one row of 130000 float32: 8.2 us, 11.7).
template <typename T>
void launch_logp_fwd_t(const LogpArgs &a, hipStream_t s) {
    const int64_t n = (a.V + kVec<T> - 1) / kVec<T>;
    if (n <= 512)
        hipLaunchKernelGGL((logp_fwd_kernel<T, 64>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
    else if (n <= 4096)
        hipLaunchKernelGGL((logp_fwd_kernel<T, 256>), dim3((unsigned)a.T), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((logp_fwd_kernel<T, 512>), dim3((unsigned)a.T), dim3(512), 0, s, a);
}

int64_t bwd_chunks(int64_t V, int ve) { return std::max<int64_t>(1, (V / ve + 1023) / 1024); }

// A wavefront to a row up to 256 vectors (16384 x 1000 bfloat16: 12.0 us, 17.6
// with a workgroup each); else a workgroup to 1024 vectors of one.
template <typename T>
void launch_logp_bwd_t(const LogpArgs &a, hipStream_t s) {
    if (a.V / kVec<T> <= 256) {
        hipLaunchKernelGGL((logp_bwd_kernel<T, 64, 4>), dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a, 1);
    } else {
        const int64_t chunks = bwd_chunks(a.V, kVec<T>);
        hipLaunchKernelGGL((logp_bwd_kernel<T, 256, 4>), dim3((unsigned)(a.T * chunks)), dim3(256), 0, s, a,
                           (int)chunks);
    }
}

// Calls f for slices of at most `rows` rows: a launch has fewer than 2^32
// threads.
template <typename F>
void for_slices(const LogpArgs &a, int64_t rows, F &&f) {
    const int64_t es = a.bf16 ? 2 : 4;
    for (int64_t t = 0; t < a.T; t += rows) {
        LogpArgs b = a;
        b.T = std::min(rows, a.T - t);
        b.z = static_cast<const char *>(a.z) + t * a.z_stride * es;
        b.dz = a.dz ? static_cast<char *>(a.dz) + t * a.dz_stride * es : nullptr;
        b.tgt = a.tgt + t;
        b.logp = a.logp ? a.logp + t : nullptr;
        b.stats = a.stats ? a.stats + 2 * t : nullptr;
        b.stats_in = a.stats_in ? a.stats_in + 2 * t : nullptr;
        b.dlogp = a.dlogp ? a.dlogp + t : nullptr;
        f(b);
    }
}
constexpr int64_t kMaxBlocks = (int64_t)1 << 22;   // of up to 512 threads

}  // namespace

hipError_t launch_logp_fwd(const LogpArgs &a, hipStream_t s) {
    for_slices(a, kMaxBlocks, [&](const LogpArgs &b) {
        b.bf16 ? launch_logp_fwd_t<bf16_t>(b, s) : launch_logp_fwd_t<float>(b, s);
    });
    return hipGetLastError();
}

hipError_t launch_logp_bwd(const LogpArgs &a, hipStream_t s) {
    const int64_t chunks = bwd_chunks(a.V, a.bf16 ? kVec<bf16_t> : kVec<float>);
    for_slices(a, kMaxBlocks / chunks, [&](const LogpArgs &b) {
        b.bf16 ? launch_logp_bwd_t<bf16_t>(b, s) : launch_logp_bwd_t<float>(b, s);
    });
    return hipGetLastError();
}

size_t policy_workspace_bytes(int64_t T, int64_t V, int bf16) {
    return ws_align((size_t)(kWeightParts + 4 * policy_blocks(T, V, bf16)) * sizeof(double));
}

hipError_t launch_policy(const PolicyArgs &a, hipStream_t s) {
    // up to kOwnWeights tokens every wavefront sums the weights for itself
    const int parts = a.T <= kOwnWeights ? 0 : (int)std::min<int64_t>(kWeightParts, (a.T + 255) / 256);
    if (a.mean && parts > 0) {
        hipLaunchKernelGGL(policy_weights_kernel, dim3(parts), dim3(256), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t blocks = policy_blocks(a.T, a.V, a.bf16);
    if (blocks > 0) {
        if (a.bf16)
            launch_policy_t<bf16_t>(a, parts, blocks, s);
        else
            launch_policy_t<float>(a, parts, blocks, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || blocks == 1) return e;
    }
    hipLaunchKernelGGL(policy_finish_kernel, dim3(1), dim3(1024), 0, s, a, parts, (int)blocks);
    return hipGetLastError();
}

}  // namespace ssm
