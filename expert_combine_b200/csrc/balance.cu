// balance.cu -- training the router gate: per-expert counts and the balance
// loss of a batch (moe_balance_loss), and the gradient of the logits from the
// loss and from the gate's top-k weights (moe_route_backward).
//
// Over the valid tokens t of sequence q, with s = sigmoid(logits):
//   p_te = s_te / S_t, S_t = sum_e s_te        c_qe = picks of expert e in q
//   P_qe = sum_t p_te                          n_q  = valid tokens of q
//   loss = coeff / Q' * sum_q E / (k n_q^2) * sum_e c_qe P_qe
//   d loss / d x_te = (g_e - sum_i g_i p_ti) * s_te (1 - s_te) / S_t,
//                     g_e = coeff / Q' * E / (k n_q^2) * c_qe
//   gate: w_j = s_j / sum_i s_i over the token's picks,
//         d x_j += w_j (1 - s_j) (dw_j - sum_i dw_i w_i)
//
// Both passes read every logit once, so DRAM bounds them (the backward pass
// also writes as much as it reads); they need 2 special-function results (2^x
// and a reciprocal) per logit.  A row of E logits stays in the registers of a
// team of warps, at most 16 a lane: one warp up to E = 512, where the row's
// sums are butterflies, then ceil(E / 512) warps that join their sums through
// shared memory at one named barrier a row.
//
// 1 - s is never formed by subtraction: with u = exp(-|x|), r = 1 / (1 + u),
// s is r or u r by the sign of x and s (1 - s) = u r^2.  A row whose sigmoids
// all but vanish (S < 1e-20: every logit below about -46) is scaled by its
// largest logit first, s ~ exp(x - max), so p keeps its value as far down as
// binary32 logits go; a row of -inf counts as p = 0.
//
// The forward pass has no floating-point atomics: a CTA's contiguous token
// range is cut at the sequence borders, each piece leaves its sums in a slot
// of its own (CTA b, sequence q: slot b + q, unique because both only grow
// along the tokens), and a second kernel adds the slots of a sequence in a
// fixed order.  Results do not depend on timing.
#include "internal.h"
#include "common.cuh"

namespace mb {

namespace {

constexpr int kBalLane = 16;                 // most logits per lane
constexpr int kBalMaxTeam = kMaxExperts / (32 * kBalLane);
constexpr int kBalWarps = 8;                 // warps of a CTA (a multiple of the team below it)
constexpr int kBalRowsPerTeam = 64;          // most rows a team adds up in one FP32 register
constexpr int kBalTargetCtas = 148 * 3;
constexpr float kBalTinySum = 1e-20f;
constexpr int kFinExperts = 32, kFinLanes = 16;   // second kernel: experts x slot lanes per CTA

struct BalPlan {
    int W;        // warps per team
    int teams;    // teams per CTA
    int nv;       // groups of 4 logits per lane
    int rows;     // rows per team
    int tokens;   // tokens per CTA
    int ctas;
};

BalPlan bal_plan(int T, int E) {
    BalPlan p;
    p.W = (E + 32 * kBalLane - 1) / (32 * kBalLane);
    p.teams = kBalWarps / p.W;
    p.nv = (E + 128 * p.W - 1) / (128 * p.W);
    int64_t rows = (static_cast<int64_t>(T) + static_cast<int64_t>(kBalTargetCtas) * p.teams - 1) /
                   (static_cast<int64_t>(kBalTargetCtas) * p.teams);
    p.rows = static_cast<int>(rows < 1 ? 1 : rows > kBalRowsPerTeam ? kBalRowsPerTeam : rows);
    p.tokens = p.rows * p.teams;
    p.ctas = T == 0 ? 1 : static_cast<int>((static_cast<int64_t>(T) + p.tokens - 1) / p.tokens);
    return p;
}

struct BalArgs {
    const float* logits;        // [T, E]
    const int32_t* ids;         // [T, k]
    const uint8_t* mask;        // [T]
    const int32_t* offsets;     // [Q + 1] or NULL (one sequence)
    int T, E, k, Q;
    int W, teams, tokens;
    float coeff;
    // forward
    float* slot_p;              // [ctas + Q][E]
    int32_t* slot_c;            // [ctas + Q][E]
    int32_t* slot_n;            // [ctas + Q]
    float* loss_part;           // [Q][experts / kFinExperts]
    unsigned int* ticket;
    float* loss;                // [1]
    int32_t* counts;            // [Q, E]
    float* prob_sums;           // [Q, E]
    int32_t* seq_tokens;        // [Q]
    // backward
    const float* grad_w;        // [T, k] or NULL
    const float* grad_loss;     // [1] or NULL
    const int32_t* counts_in;
    const int32_t* seq_tokens_in;
    float* grad;                // [T, E]
};

__device__ __forceinline__ float ex2_approx(float t) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return e;
}
__device__ __forceinline__ float rcp_approx(float t) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// Expert of element i of this lane: groups of 4 in a row (VEC, E % 4 == 0) or
// a stride of 32 (any E).
template <int NV, bool VEC>
__device__ __forceinline__ int bal_expert(int wt, int lane, int i) {
    return VEC ? (wt * NV + (i >> 2)) * 128 + lane * 4 + (i & 3) : wt * NV * 128 + i * 32 + lane;
}

// One row's logits of this lane; elements past E read as -inf (sigmoid 0).
template <int NV, bool VEC>
__device__ __forceinline__ void bal_load(const float* row, int E, int wt, int lane, float (&x)[4 * NV]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if constexpr (VEC) {
            const int e = bal_expert<NV, VEC>(wt, lane, 4 * v);
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < E) f = ld_nc_f4(row + e);
            x[4 * v] = f.x, x[4 * v + 1] = f.y, x[4 * v + 2] = f.z, x[4 * v + 3] = f.w;
        } else {
#pragma unroll
            for (int i = 4 * v; i < 4 * v + 4; ++i) {
                const int e = bal_expert<NV, VEC>(wt, lane, i);
                x[i] = e < E ? __ldg(row + e) : -INFINITY;
            }
        }
    }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Joins the team's per-warp values: one barrier, two alternating buffers.
struct Team {
    float2* red;     // [2][kBalMaxTeam]
    int W, bar, wt, lane;
    int par;
    __device__ __forceinline__ float2 sum(float2 v) {
        v.x = warp_tree_sum(v.x);
        v.y = warp_tree_sum(v.y);
        return join<false>(v);
    }
    __device__ __forceinline__ float sum(float v) { return join<false>(make_float2(warp_tree_sum(v), 0.0f)).x; }
    __device__ __forceinline__ float max(float v) { return join<true>(make_float2(warp_max(v), 0.0f)).x; }
    template <bool MAX>
    __device__ __forceinline__ float2 join(float2 v) {
        if (W == 1) {
            __syncwarp();
            return v;
        }
        float2* buf = red + par * kBalMaxTeam;
        par ^= 1;
        if (lane == 0) buf[wt] = v;
        named_bar_sync(bar, W * 32);
        float2 a = buf[0];
        for (int w = 1; w < W; ++w) {
            a.x = MAX ? fmaxf(a.x, buf[w].x) : a.x + buf[w].x;
            a.y += buf[w].y;
        }
        return a;
    }
};

__device__ __forceinline__ int clamp_offset(const BalArgs& a, int q) {
    if (a.offsets == nullptr) return q == 0 ? 0 : a.T;
    const int o = a.offsets[q];
    return o < 0 ? 0 : o > a.T ? a.T : o;
}

// First sequence that ends behind token t (Q when none does).
__device__ __forceinline__ int first_sequence(const BalArgs& a, int t) {
    int lo = 0, hi = a.Q;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (clamp_offset(a, mid + 1) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

template <int NV, bool VEC>
__global__ void __launch_bounds__(kBalWarps * 32) balance_kernel(const BalArgs a) {
    constexpr int NE = 4 * NV;
    extern __shared__ __align__(16) uint8_t bal_smem[];
    float* sums = reinterpret_cast<float*>(bal_smem);                    // [teams][E]
    int32_t* hist = reinterpret_cast<int32_t*>(sums + a.teams * a.E);    // [E]
    __shared__ float2 red[kBalWarps][2 * kBalMaxTeam];
    __shared__ int s_n;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / a.W;
    Team tm{red[team], a.W, 1 + team, warp % a.W, lane, 0};
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    const int t1 = static_cast<int>(min(t0 + a.tokens, static_cast<int64_t>(a.T)));

    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    if (threadIdx.x == 0) s_n = 0;
    griddep_wait();
    griddep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
    __syncthreads();

    for (int q = first_sequence(a, static_cast<int>(t0)); q < a.Q; ++q) {
        const int lo = clamp_offset(a, q);
        if (lo >= t1) break;
        const int s = max(static_cast<int>(t0), lo), e_ = min(t1, clamp_offset(a, q + 1));
        if (s >= e_) continue;

        float acc[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = 0.0f;
        int n = 0;
        float x[NE];
        bool valid = false;
        int id = -1;
        auto fetch = [&](int t, float (&xx)[NE], bool& v, int& d) {
            v = false;
            if (t < e_) {
                bal_load<NV, VEC>(a.logits + static_cast<size_t>(t) * a.E, a.E, tm.wt, lane, xx);
                v = a.mask[t] != 0;
                if (tm.wt == 0) d = lane < a.k ? a.ids[static_cast<size_t>(t) * a.k + lane] : -1;
            }
        };
        fetch(s + team, x, valid, id);
        for (int t = s + team; t < e_; t += a.teams) {
            float xn[NE];
            bool nvalid;
            int nid = -1;
            fetch(t + a.teams, xn, nvalid, nid);
            if (valid) {
                float loc = 0.0f;
                float sg[NE];
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    sg[i] = rcp_approx(1.0f + ex2_approx(x[i] * -kLog2e));
                    loc += sg[i];
                }
                float S = tm.sum(loc);
                if (S < kBalTinySum) {
                    float m = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NE; ++i) m = fmaxf(m, x[i]);
                    m = tm.max(m);
                    loc = 0.0f;
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        sg[i] = m == -INFINITY ? 0.0f : ex2_approx((x[i] - m) * kLog2e);
                        loc += sg[i];
                    }
                    S = tm.sum(loc);
                }
                const float inv = S == 0.0f ? 0.0f : __frcp_rn(S);
#pragma unroll
                for (int i = 0; i < NE; ++i) acc[i] = fmaf(sg[i], inv, acc[i]);
                if (tm.wt == 0) {
                    if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
                    ++n;
                }
            }
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = xn[i];
            valid = nvalid;
            id = nid;
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = bal_expert<NV, VEC>(tm.wt, lane, i);
            if (e < a.E) sums[team * a.E + e] = acc[i];
        }
        if (tm.wt == 0 && lane == 0 && n) atomicAdd(&s_n, n);
        __syncthreads();
        const size_t slot = static_cast<size_t>(blockIdx.x) + q;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float p = sums[e];
            for (int m = 1; m < a.teams; ++m) p += sums[m * a.E + e];
            a.slot_p[slot * a.E + e] = p;
            a.slot_c[slot * a.E + e] = hist[e];
            hist[e] = 0;
        }
        if (threadIdx.x == 0) {
            a.slot_n[slot] = s_n;
            s_n = 0;
        }
        __syncthreads();
    }
}

// Adds a sequence's slots (kFinLanes runs of them, then the runs in order) and
// writes its outputs; the last CTA to finish adds the losses.
__global__ void __launch_bounds__(kFinExperts * kFinLanes) balance_finish_kernel(const BalArgs a, int parts) {
    __shared__ float sp[kFinLanes][kFinExperts];
    __shared__ int sc[kFinLanes][kFinExperts];
    __shared__ int s_n;
    __shared__ bool s_last;
    __shared__ double s_loss[kFinLanes];
    __shared__ int s_some;
    const int el = threadIdx.x % kFinExperts, sl = threadIdx.x / kFinExperts;
    const int e = blockIdx.x * kFinExperts + el;
    if (threadIdx.x == 0) s_n = 0, s_some = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch();
    for (int q = blockIdx.y; q < a.Q; q += gridDim.y) {
        const int lo = clamp_offset(a, q), hi = clamp_offset(a, q + 1);
        float p = 0.0f;
        int c = 0, n = 0;
        if (lo < hi) {
            const int b0 = lo / a.tokens, b1 = (hi - 1) / a.tokens;
            for (int b = b0 + sl; b <= b1; b += kFinLanes) {
                const size_t slot = static_cast<size_t>(b) + q;
                if (e < a.E) {
                    p += a.slot_p[slot * a.E + e];
                    c += a.slot_c[slot * a.E + e];
                }
                if (el == 0) n += a.slot_n[slot];
            }
        }
        sp[sl][el] = p;
        sc[sl][el] = c;
        if (n) atomicAdd(&s_n, n);
        __syncthreads();
        if (sl == 0) {
            for (int m = 1; m < kFinLanes; ++m) {
                p += sp[m][el];
                c += sc[m][el];
            }
            n = s_n;
            if (e < a.E) {
                a.prob_sums[static_cast<size_t>(q) * a.E + e] = p;
                a.counts[static_cast<size_t>(q) * a.E + e] = c;
            }
            // a sequence without a valid token adds nothing
            const float dot = warp_tree_sum(n > 0 && e < a.E ? static_cast<float>(c) * p : 0.0f);
            if (el == 0) {
                const float fn = static_cast<float>(n);
                a.loss_part[static_cast<size_t>(q) * parts + blockIdx.x] =
                    n > 0 ? dot * (static_cast<float>(a.E) / static_cast<float>(a.k)) / fn / fn : 0.0f;
                if (blockIdx.x == 0) a.seq_tokens[q] = n;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(a.ticket, 1u) == gridDim.x * gridDim.y - 1;
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    double l = 0.0;
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(a.Q) * parts; i += blockDim.x) l += __ldcg(a.loss_part + i);
    int some = 0;
    for (int q = threadIdx.x; q < a.Q; q += blockDim.x) some += __ldcg(a.seq_tokens + q) > 0;
    if (some) atomicAdd(&s_some, some);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (el == 0) s_loss[sl] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int m = 1; m < kFinLanes; ++m) l += s_loss[m];
        a.loss[0] = static_cast<float>(l * a.coeff / (s_some > 0 ? s_some : 1));
    }
}

// The gradient of the logits.  A team keeps its row in registers; the few
// entries of the gate's own gradient are laid into a row of shared memory
// (zero elsewhere) that the dense pass adds, so every logit's gradient is
// written once, in full lines.
template <int NV, bool VEC, bool BAL>
__global__ void __launch_bounds__(kBalWarps * 32) gate_grad_kernel(const BalArgs a) {
    constexpr int NE = 4 * NV;
    extern __shared__ __align__(16) uint8_t bal_smem[];
    __shared__ float2 red[kBalWarps][2 * kBalMaxTeam];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / a.W;
    const int pitch = (a.E + 3) & ~3;
    float* add0 = reinterpret_cast<float*>(bal_smem) + static_cast<size_t>(team) * 2 * pitch;   // two rows per team
    Team tm{red[team], a.W, 1 + team, warp % a.W, lane, 0};
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    const int t1 = static_cast<int>(min(t0 + a.tokens, static_cast<int64_t>(a.T)));
    for (int e = threadIdx.x; e < a.teams * 2 * pitch; e += blockDim.x) reinterpret_cast<float*>(bal_smem)[e] = 0.0f;
    griddep_wait();
    griddep_launch();
    float unit = 0.0f;
    if constexpr (BAL) {
        __shared__ int s_some;
        if (threadIdx.x == 0) s_some = 0;
        __syncthreads();
        int some = 0;
        for (int q = threadIdx.x; q < a.Q; q += blockDim.x) some += a.seq_tokens_in[q] > 0;
        if (some) atomicAdd(&s_some, some);
        __syncthreads();
        unit = a.grad_loss[0] * a.coeff * (static_cast<float>(a.E) / static_cast<float>(a.k)) /
               static_cast<float>(s_some > 0 ? s_some : 1);
    } else {
        __syncthreads();
    }

    int q = BAL ? first_sequence(a, static_cast<int>(t0)) : a.Q;
    int q_of_g = -1;
    float g[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) g[i] = 0.0f;
    int old_id = -1;
    int par = 0;
    for (int t = static_cast<int>(t0) + team; t < t1; t += a.teams, par ^= 1) {
        float* add = add0 + par * pitch;
        const bool valid = a.mask[t] != 0;
        bool in_seq = false;
        float x[NE];
        if constexpr (BAL) {
            if (valid) {
                bal_load<NV, VEC>(a.logits + static_cast<size_t>(t) * a.E, a.E, tm.wt, lane, x);
                while (q < a.Q && clamp_offset(a, q + 1) <= t) ++q;
                in_seq = q < a.Q && clamp_offset(a, q) <= t;
                if (in_seq && q != q_of_g) {
                    q_of_g = q;
                    const int n = a.seq_tokens_in[q];
                    const float fn = static_cast<float>(n);
                    const float c = n > 0 ? unit / fn / fn : 0.0f;
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        const int e = bal_expert<NV, VEC>(tm.wt, lane, i);
                        g[i] = e < a.E ? c * static_cast<float>(a.counts_in[static_cast<size_t>(q) * a.E + e]) : 0.0f;
                    }
                }
            }
        }
        // the gate's own gradient: one pick per lane
        int id = -1;
        if (tm.wt == 0 && a.grad_w != nullptr && valid) {
            float xj = -INFINITY, dw = 0.0f;
            if (lane < a.k) {
                id = a.ids[static_cast<size_t>(t) * a.k + lane];
                if (id < 0 || id >= a.E) id = -1;
                if (id >= 0) {
                    xj = a.logits[static_cast<size_t>(t) * a.E + id];
                    dw = a.grad_w[static_cast<size_t>(t) * a.k + lane];
                }
            }
            const float m = fminf(warp_max(xj), 0.0f);
            const float u = expf(-fabsf(xj)), r = __frcp_rn(1.0f + u);
            // s exp(-m): sigmoids relative to the largest, 1 - s from the same two
            const float sj = xj == -INFINITY ? 0.0f : expf(fminf(xj, 0.0f) - m) * r;
            const float tot = warp_tree_sum(sj);
            const float w = tot == 0.0f ? 0.0f : __fdiv_rn(sj, tot);
            const float dot = warp_tree_sum(dw * w);
            float d = w * (xj >= 0.0f ? u * r : r) * (dw - dot);
            const unsigned same = __match_any_sync(0xffffffffu, id);
            if (__any_sync(0xffffffffu, id >= 0 && __popc(same) > 1)) {   // the same expert twice: added in slot order
                float z = 0.0f;
                for (int j = 0; j < 32; ++j) {
                    const float dj = __shfl_sync(0xffffffffu, d, j);
                    if (same >> j & 1u) z += dj;
                }
                d = z;
            }
            __syncwarp();   // behind the lanes that cleared this buffer
            if (id >= 0) add[id] = d;
        }
        float S = 0.0f, G = 0.0f;
        float sl[NE];
        if (BAL && in_seq) {
            float2 loc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const float u = ex2_approx(fabsf(x[i]) * -kLog2e), r = rcp_approx(1.0f + u), ur = u * r;
                const float s = x[i] >= 0.0f ? r : ur;
                sl[i] = ur * r;
                loc.x += s;
                loc.y = fmaf(g[i], s, loc.y);
            }
            loc = tm.sum(loc);
            if (loc.x < kBalTinySum) {
                float m = -INFINITY;
#pragma unroll
                for (int i = 0; i < NE; ++i) m = fmaxf(m, x[i]);
                m = tm.max(m);
                loc = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    sl[i] = m == -INFINITY ? 0.0f : ex2_approx((x[i] - m) * kLog2e);
                    loc.x += sl[i];
                    loc.y = fmaf(g[i], sl[i], loc.y);
                }
                loc = tm.sum(loc);
            }
            S = loc.x == 0.0f ? 0.0f : __frcp_rn(loc.x);
            G = loc.y * S;
        } else {
            tm.sum(0.0f);   // the barrier that makes `add` visible to the team
        }
        // the previous row's entries: every warp has read them by now
        if (old_id >= 0) (add0 + (par ^ 1) * pitch)[old_id] = 0.0f;
        old_id = id;
        float* row = a.grad + static_cast<size_t>(t) * a.E;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = BAL && in_seq ? (g[4 * v + i] - G) * (sl[4 * v + i] * S) : 0.0f;
            if constexpr (VEC) {
                const int e = bal_expert<NV, VEC>(tm.wt, lane, 4 * v);
                if (e < a.E) {
                    const float4 z = *reinterpret_cast<const float4*>(add + e);
                    __stcs(reinterpret_cast<float4*>(row + e),
                           make_float4(d[0] + z.x, d[1] + z.y, d[2] + z.z, d[3] + z.w));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = bal_expert<NV, VEC>(tm.wt, lane, 4 * v + i);
                    if (e < a.E) __stcs(row + e, d[i] + add[e]);
                }
            }
        }
    }
}

template <typename F>
cudaError_t bal_launch(F* kernel, const BalPlan& p, size_t smem, const BalArgs& a, cudaStream_t s) {
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas);
    cfg.blockDim = dim3(p.W * p.teams * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool VEC>
cudaError_t launch_balance_main(const BalPlan& p, size_t smem, const BalArgs& a, cudaStream_t s) {
    switch (p.nv) {
        case 1: return bal_launch(balance_kernel<1, VEC>, p, smem, a, s);
        case 2: return bal_launch(balance_kernel<2, VEC>, p, smem, a, s);
        case 3: return bal_launch(balance_kernel<3, VEC>, p, smem, a, s);
        default: return bal_launch(balance_kernel<4, VEC>, p, smem, a, s);
    }
}
template <bool VEC, bool BAL>
cudaError_t launch_gate_grad(const BalPlan& p, size_t smem, const BalArgs& a, cudaStream_t s) {
    switch (p.nv) {
        case 1: return bal_launch(gate_grad_kernel<1, VEC, BAL>, p, smem, a, s);
        case 2: return bal_launch(gate_grad_kernel<2, VEC, BAL>, p, smem, a, s);
        case 3: return bal_launch(gate_grad_kernel<3, VEC, BAL>, p, smem, a, s);
        default: return bal_launch(gate_grad_kernel<4, VEC, BAL>, p, smem, a, s);
    }
}

size_t pad16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }
int bal_parts(int E) { return (E + kFinExperts - 1) / kFinExperts; }

}  // namespace

size_t balance_workspace_bytes(int T, int E, int Q) {
    const size_t slots = static_cast<size_t>(bal_plan(T, E).ctas) + Q;
    return 16 + 2 * pad16(slots * E * 4) + pad16(slots * 4) + pad16(static_cast<size_t>(Q) * bal_parts(E) * 4);
}

cudaError_t launch_balance_loss(const BalanceLaunch& b, cudaStream_t s) {
    const BalPlan p = bal_plan(b.T, b.E);
    BalArgs a{};
    a.logits = b.logits, a.ids = b.ids, a.mask = b.mask, a.offsets = b.offsets;
    a.T = b.T, a.E = b.E, a.k = b.k, a.Q = b.Q, a.coeff = b.coeff;
    a.W = p.W, a.teams = p.teams, a.tokens = p.tokens;
    const size_t slots = static_cast<size_t>(p.ctas) + b.Q;
    uint8_t* w = static_cast<uint8_t*>(b.workspace);
    a.ticket = reinterpret_cast<unsigned int*>(w);
    a.slot_p = reinterpret_cast<float*>(w += 16);
    a.slot_c = reinterpret_cast<int32_t*>(w += pad16(slots * b.E * 4));
    a.slot_n = reinterpret_cast<int32_t*>(w += pad16(slots * b.E * 4));
    a.loss_part = reinterpret_cast<float*>(w += pad16(slots * 4));
    a.loss = b.loss, a.counts = b.counts, a.prob_sums = b.prob_sums, a.seq_tokens = b.seq_tokens;
    const size_t smem = static_cast<size_t>(p.teams + 1) * b.E * 4;
    cudaError_t e = b.E % 4 == 0 ? launch_balance_main<true>(p, smem, a, s) : launch_balance_main<false>(p, smem, a, s);
    if (e != cudaSuccess) return e;
    const int parts = bal_parts(b.E);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts, b.Q < 65535 ? b.Q : 65535);
    cfg.blockDim = dim3(kFinExperts * kFinLanes);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, balance_finish_kernel, a, parts);
}

cudaError_t launch_route_backward(const GateGradLaunch& b, cudaStream_t s) {
    const BalPlan p = bal_plan(b.T, b.E);
    BalArgs a{};
    a.logits = b.logits, a.ids = b.ids, a.mask = b.mask, a.offsets = b.offsets;
    a.T = b.T, a.E = b.E, a.k = b.k, a.Q = b.Q, a.coeff = b.coeff;
    a.W = p.W, a.teams = p.teams, a.tokens = p.tokens;
    a.grad_w = b.grad_w, a.grad_loss = b.grad_loss, a.counts_in = b.counts, a.seq_tokens_in = b.seq_tokens;
    a.grad = b.grad;
    const size_t smem = static_cast<size_t>(p.teams) * 2 * ((b.E + 3) & ~3) * 4;
    const bool bal = b.grad_loss != nullptr;
    if (b.E % 4 == 0) return bal ? launch_gate_grad<true, true>(p, smem, a, s) : launch_gate_grad<true, false>(p, smem, a, s);
    return bal ? launch_gate_grad<false, true>(p, smem, a, s) : launch_gate_grad<false, false>(p, smem, a, s);
}

}  // namespace mb
