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
// also writes as much as it reads); they need 3 special-function results for two
// logits (two 2^x and a shared reciprocal).  A row of E logits belongs to a team of warps, at
// most 16 logits a lane: one warp up to E = 512, where the row's sums are
// butterflies, then ceil(E / 512) warps that join their sums through shared
// memory at one named barrier a row.  Each warp streams its part of the team's
// rows through a ring of its own in shared memory, filled by bulk copies that
// its lane 0 starts up to 8 rows ahead, so loads need neither registers nor
// warps in waiting (rows of E % 4 != 0 are read one ahead into registers).
//
// 1 - s is never formed by subtraction: s (1 - s) = exp(-x) s^2.  A row whose
// sigmoids all but vanish (S < 1e-6) or whose exponentials leave the range is
// done over relative to its largest logit, so p keeps its value as far down as
// binary32 logits go, and -inf (an expert shut out) has p = 0 and no gradient.
//
// The forward pass has no floating-point atomics: a CTA's contiguous token
// range is cut at the sequence borders, each piece leaves its sums in a slot
// of its own (CTA b, sequence q: slot b + q, unique because both only grow
// along the tokens), and a second kernel adds the slots of a sequence in a
// fixed order.  A small batch runs as one cluster of 8 CTAs whose slots are
// their shared memory: one launch, no workspace.  Results do not depend on
// timing.
//
// From a graph, 65536 x 512, k = 22: loss 36 us (floor at the copy rate 21),
// gradient 73 us (43); 32768 x 2560, k = 8: 82 us (51) and 133 us (103; called
// one by one 138).
#include "internal.h"
#include "common.cuh"

namespace mb {

namespace {

constexpr int kBalLane = 16;                 // most logits per lane
constexpr int kBalMaxTeam = kMaxExperts / (32 * kBalLane);
constexpr int kBalWarps = 24;                // most warps of a CTA (one CTA per SM): the loss
constexpr int kBalGradWarps = 16;            // of the gradient, which needs twice the registers, and of a cluster's CTAs
constexpr int kBalGateWarps = 4;             // warps of the gradient for the gate's own part
static_assert(kBalGradWarps <= 4 * kBalGateWarps, "a gate warp serves four teams at most");
static_assert(kBalWarps / 2 <= 15 && kBalGradWarps / 2 <= 15, "a team of several warps has a hardware barrier of its own, 1 .. 15");
constexpr int kBalTags = 1024;               // marks per row for finding repeated picks
constexpr int kBalLists = 4;                 // lists of entries a team has under way
constexpr int kBalRowsPerTeam = 128;         // most rows a team adds up in one FP32 register
constexpr int kBalTargetCtas = 148;
constexpr int kBalRing = 8;                  // most row slots of a warp
constexpr int kBalRingBytes = 128 * 1024;    // of a CTA
// A row's sigmoids are summed plainly while their sum is at least kBalTinySum.
// What stands behind the row's end (kBalPast) adds 4e-18 a place to it.
constexpr float kBalTinySum = 1e-6f;
constexpr float kBalPast = -40.0f;
constexpr unsigned int kBalTimeout = 64u;    // bit 6 of the device status word
constexpr int kFinExperts = 32, kFinLanes = 16;   // second kernel: experts x slot lanes per CTA
constexpr int kBalCluster = 8;               // small batches: CTAs of the one cluster
constexpr int kBalClusterLogits = 256 * 1024;     // T * E up to here (1 MB of logits through 8 SMs)
constexpr int kBalClusterRows = 32;               // rows a team takes at most
constexpr int kBalClusterSums = 4096;             // Q * E up to here (32 KB of shared memory)

struct BalPlan {
    int W;        // warps per team
    int teams;    // teams per CTA
    int nv;       // groups of 4 logits per lane
    int tokens;   // tokens per CTA
    int ctas;
    int ring;     // row slots per warp
    bool cluster; // forward pass in one cluster
};

// Lanes per row of picks.
__host__ __device__ __forceinline__ int bal_group(int k) { return k <= 8 ? 8 : k <= 16 ? 16 : 32; }

BalPlan bal_plan(int T, int E, int Q, bool grad) {
    BalPlan p;
    p.W = (E + 32 * kBalLane - 1) / (32 * kBalLane);
    p.nv = (E + 128 * p.W - 1) / (128 * p.W);
    p.cluster = !grad && T <= kBalCluster * (kBalGradWarps / p.W) * kBalClusterRows &&
                static_cast<int64_t>(T) * E <= kBalClusterLogits && static_cast<int64_t>(Q) * E <= kBalClusterSums;
    p.teams = (grad || p.cluster ? kBalGradWarps : kBalWarps) / p.W;
    const int64_t ctas = p.cluster ? kBalCluster : kBalTargetCtas;
    // as many rows a team as fill the card's teams, in several waves where that were more than kBalRowsPerTeam
    const int64_t per = ctas * p.teams;
    const int64_t waves = T == 0 ? 1 : (T + per * kBalRowsPerTeam - 1) / (per * kBalRowsPerTeam);
    int64_t rows = (T + per * waves - 1) / (per * waves);
    if (rows < 1) rows = 1;
    p.tokens = static_cast<int>(rows) * p.teams;
    p.ctas = T == 0 ? 1 : static_cast<int>((static_cast<int64_t>(T) + p.tokens - 1) / p.tokens);
    p.ring = 0;
    if (E % 4 == 0) {
        p.ring = kBalRingBytes / (p.W * p.teams * p.nv * 512);
        if (p.ring > kBalRing) p.ring = kBalRing;
        if (p.ring > rows) p.ring = static_cast<int>(rows);
    }
    return p;
}

struct BalArgs {
    const float* logits;        // [T, E]
    const int32_t* ids;         // [T, k]
    const uint8_t* mask;        // [T]
    const int32_t* offsets;     // [Q + 1] or NULL (one sequence)
    int T, E, k, Q;
    int W, teams, tokens, ring;
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
// Store to `local`'s place in the shared memory of cluster rank `rank`.
__device__ __forceinline__ void st_cluster(float* local, uint32_t rank, float v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
}
constexpr float kLog2e = 1.4426950408889634f;

// The sigmoids of two logits, e their exponentials exp(-x).  One reciprocal
// serves both, 1 / a = b / (a b): the special-function unit, which bounds these
// kernels next to DRAM, forms 3 results for a pair instead of 4.  `big` grows
// to infinity where a b leaves the range in which its reciprocal is normal (the
// pair's logits, those above 0 taken for 0, add up to less than -87); the row
// is then done over by sigmoid_over.
__device__ __forceinline__ float2 sigmoid2(float2 x, float2& e, float& big) {
    const float2 t = mul2(x, make_float2(-kLog2e, -kLog2e));
    e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    const float2 d = add2(e, make_float2(1.0f, 1.0f));
    const float p = d.x * d.y, q = rcp_approx(p);
    big = fmaf(p, 4.0f, big);
    return make_float2(q * d.y, q * d.x);
}

// For any row: sigmoid(x) / exp(min(m, 0)) with m the row's largest logit, and
// that times 1 - sigmoid(x).  With u = exp(-|x|), r = 1 / (1 + u) the sigmoid is
// exp(min(x, 0)) r and 1 - sigmoid u r or r by the sign of x.  A logit of -inf
// gives 0, also in a row of nothing else; NaN gives NaN whatever m is (fmaxf
// leaves NaN out of m, so a row of NaN and -inf has m = -inf).
__device__ __forceinline__ float sigmoid_over(float x, float m, float& slope) {
    const float u = ex2_approx(fabsf(x) * -kLog2e), r = rcp_approx(1.0f + u);
    const float s = x == -INFINITY ? 0.0f : ex2_approx((fminf(x, 0.0f) - fminf(m, 0.0f)) * kLog2e) * r;
    slope = s * (x >= 0.0f ? u * r : r);
    return s;
}

// Expert of element i of this lane: groups of 4 in a row (VEC, E % 4 == 0) or
// a stride of 32 (any E).
template <int NV, bool VEC>
__device__ __forceinline__ int bal_expert(int wt, int lane, int i) {
    return VEC ? (wt * NV + (i >> 2)) * 128 + lane * 4 + (i & 3) : wt * NV * 128 + i * 32 + lane;
}

// One row's logits of this lane; `past` stands for elements behind E.
template <int NV, bool VEC>
__device__ __forceinline__ void bal_load(const float* row, int E, int wt, int lane, float past, float (&x)[4 * NV]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if constexpr (VEC) {
            const int e = bal_expert<NV, VEC>(wt, lane, 4 * v);
            float4 f = make_float4(past, past, past, past);
            if (e < E) f = ld_nc_f4(row + e);
            x[4 * v] = f.x, x[4 * v + 1] = f.y, x[4 * v + 2] = f.z, x[4 * v + 3] = f.w;
        } else {
#pragma unroll
            for (int i = 4 * v; i < 4 * v + 4; ++i) {
                const int e = bal_expert<NV, VEC>(wt, lane, i);
                x[i] = e < E ? __ldg(row + e) : past;
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
#pragma unroll
        for (int w = 1; w < kBalMaxTeam; ++w) {
            if (w >= W) break;
            const float2 o = buf[w];
            a.x = MAX ? fmaxf(a.x, o.x) : a.x + o.x;
            a.y += o.y;
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

// This warp's part of its team's rows (tokens first, first + teams, ...), in
// order, as pairs of logits.
template <int NV, bool VEC>
struct RowFeed {
    const float* next;       // VEC: the warp's part of the next row to copy; else of the next row to read
    size_t pitch;            // floats from row to row
    int left;                // rows not yet copied (VEC) or read
    int flying;              // rows copied or being copied, not yet taken
    int slot, phase, ring, bytes, lane, wt, E;
    float* slots;
    uint64_t* full;
    bool dead;
    float ahead[VEC ? 1 : 4 * NV];

    __device__ __forceinline__ void start(const BalArgs& a, const Team& tm, int warp, int first, int end, uint8_t* smem,
                                          uint64_t* bars) {
        lane = tm.lane, wt = tm.wt, E = a.E, ring = a.ring, slot = 0, phase = 0, flying = 0, dead = false;
        left = first < end ? (end - first + a.teams - 1) / a.teams : 0;
        pitch = static_cast<size_t>(a.teams) * a.E;
        next = a.logits + static_cast<size_t>(first) * a.E;
        if constexpr (VEC) {
            next += wt * NV * 128;
            slots = reinterpret_cast<float*>(smem) + static_cast<size_t>(warp) * ring * NV * 128;
            full = bars + warp * kBalRing;
            const int mine = E - wt * NV * 128;
            bytes = 4 * (mine < 0 ? 0 : mine < NV * 128 ? mine : NV * 128);
            if (bytes < NV * 512) {     // behind the row's end the copies write nothing
                for (int i = lane; i < ring * NV * 128; i += 32) slots[i] = kBalPast;
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (bytes == 0) left = 0;
            for (int i = 0; i < ring && left > 0; ++i) {
                if (lane == 0) copy(i);
                advance();
            }
        } else {
            if (left > 0) bal_load<NV, VEC>(next, E, wt, lane, kBalPast, ahead);
        }
    }
    __device__ __forceinline__ void copy(int s) {
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(bytes));
        bulk_g2s(slots + s * NV * 128, next, static_cast<uint32_t>(bytes), &full[s]);
    }
    __device__ __forceinline__ void advance() {
        next += pitch;
        --left;
        ++flying;
    }
    // The next row.
    __device__ __forceinline__ void take(float2 (&x)[2 * NV]) {
        if constexpr (VEC) {
            // After a wait that ran out the values are not the row's, but the team keeps its barriers.  Every lane
            // polls, and the warp takes it for run out together where it ran out in one of them, so that the
            // lanes go on agreeing about what is in flight.
            if (flying > 0 && !dead)
                dead = __any_sync(0xffffffffu,
                                  !mbar_wait_bounded(&full[slot], static_cast<uint32_t>(phase), kBalTimeout));
            const float* p = slots + slot * NV * 128 + 4 * lane;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float4 f = *reinterpret_cast<const float4*>(p + 128 * v);
                x[2 * v] = make_float2(f.x, f.y), x[2 * v + 1] = make_float2(f.z, f.w);
            }
            if (flying > 0) {
                --flying;
                __syncwarp();      // every lane has its values: the slot is free
                if (left > 0 && !dead) {
                    if (lane == 0) {
                        fence_proxy_async_smem();
                        copy(slot);
                    }
                    advance();
                }
                if (++slot == ring) slot = 0, phase ^= 1;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2 * NV; ++i) x[i] = make_float2(ahead[2 * i], ahead[2 * i + 1]);
            next += pitch;
            if (--left > 0) bal_load<NV, VEC>(next, E, wt, lane, kBalPast, ahead);
        }
    }
    // Copies that were started and not used land before the CTA ends.
    __device__ __forceinline__ void drain() {
        if constexpr (VEC)
            if (lane == 0)
                for (; flying > 0; --flying) {
                    mbar_wait_bounded(&full[slot], static_cast<uint32_t>(phase), kBalTimeout);
                    if (++slot == ring) slot = 0, phase ^= 1;
                }
    }
};

// Which of a team's rows are valid tokens, 32 rows at a time (one byte a lane),
// the next 32 already on their way.
struct RowMask {
    const uint8_t* p;        // this lane's next byte
    int64_t t, end, step;
    uint32_t bits, byte;
    int at;
    __device__ __forceinline__ void start(const BalArgs& a, int lane, int first, int last) {
        step = 32 * static_cast<int64_t>(a.teams);
        t = first + static_cast<int64_t>(lane) * a.teams;
        end = last;
        p = a.mask + t;
        at = 32;
        fetch();
    }
    __device__ __forceinline__ void fetch() {
        byte = t < end ? *p : 0;
        t += step;
        p += step;
    }
    __device__ __forceinline__ bool next() {
        if (at == 32) {
            bits = __ballot_sync(0xffffffffu, byte != 0);
            at = 0;
            fetch();
        }
        return bits >> at++ & 1u;
    }
};

// Shared memory of the CTA: the warps' rings, then what the kernel adds.
template <int NV>
__host__ __device__ __forceinline__ size_t bal_ring_bytes(int warps, int ring) {
    return static_cast<size_t>(warps) * ring * NV * 512;
}

// CL: one cluster of kBalCluster CTAs does all; the slots are shared memory.
template <int NV, bool VEC, bool CL>
__global__ void __launch_bounds__((CL ? kBalGradWarps : kBalWarps) * 32, 1) balance_kernel(const BalArgs a) {
    constexpr int NE = 4 * NV;
    constexpr int kWarps = CL ? kBalGradWarps : kBalWarps;
    extern __shared__ __align__(128) uint8_t bal_smem[];
    float* sums = reinterpret_cast<float*>(bal_smem + bal_ring_bytes<NV>(a.W * a.teams, a.ring));   // [teams][E]
    int32_t* hist = reinterpret_cast<int32_t*>(sums + a.teams * a.E);    // [E]
    float* own_p = reinterpret_cast<float*>(hist + a.E);                 // CL: [Q][E]
    int32_t* own_c = reinterpret_cast<int32_t*>(own_p + a.Q * a.E);      // CL: [Q][E]
    int32_t* own_n = own_c + a.Q * a.E;                                  // CL: [Q]
    float* own_l = reinterpret_cast<float*>(own_n + a.Q);                // CL: [Q] losses (rank 0)
    __shared__ float2 red[kWarps][2 * kBalMaxTeam];
    __shared__ __align__(8) uint64_t bars[kWarps * kBalRing];
    __shared__ int s_n;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / a.W;
    Team tm{red[team], a.W, 1 + team, warp % a.W, lane, 0};
    for (int i = threadIdx.x; i < kWarps * kBalRing; i += blockDim.x) mbar_init(&bars[i], 1);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    if (CL)
        for (int i = threadIdx.x; i < a.Q * (2 * a.E + 2); i += blockDim.x) own_c[i - a.Q * a.E] = 0;
    if (threadIdx.x == 0) s_n = 0;
    fence_mbar_init();
    griddep_wait();
    griddep_launch();
    if (!CL && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
    __syncthreads();

    // this CTA's tokens that belong to a sequence
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    const int t0 = max(static_cast<int>(min(c0, static_cast<int64_t>(a.T))), clamp_offset(a, 0));
    const int t1 = min(static_cast<int>(min(c0 + a.tokens, static_cast<int64_t>(a.T))), clamp_offset(a, a.Q));
    RowFeed<NV, VEC> feed;
    feed.start(a, tm, warp, t0 + team, t1, bal_smem, bars);
    RowMask mask;
    mask.start(a, lane, t0 + team, t1);
    int t = t0 + team;
    const bool counts = tm.wt == 0 && lane < a.k;
    const int32_t* pick = a.ids + static_cast<size_t>(t < t1 ? t : 0) * a.k + lane;
    const size_t pick_step = static_cast<size_t>(a.teams) * a.k;
    int id = counts && t < t1 ? *pick : -1, id1 = counts && t + a.teams < t1 ? pick[pick_step] : -1;   // two rows ahead
    pick += 2 * pick_step;

    for (int q = first_sequence(a, t0); t0 < t1 && q < a.Q; ++q) {
        const int lo = clamp_offset(a, q), hi = min(t1, clamp_offset(a, q + 1));
        if (lo >= t1) break;
        if (max(t0, lo) >= hi) continue;

        float2 acc[NE / 2];
#pragma unroll
        for (int i = 0; i < NE / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
        int n = 0;
        for (; t < hi; t += a.teams) {
            float2 x[NE / 2];
            feed.take(x);
            const bool valid = mask.next();
            const int id2 = counts && t + 2 * a.teams < t1 ? *pick : -1;
            pick += pick_step;
            if (valid && t >= lo) {
                float2 loc = make_float2(0.0f, 0.0f);
                float big = 0.0f;
#pragma unroll
                for (int i = 0; i < NE / 2; ++i) {
                    float2 e;
                    x[i] = sigmoid2(x[i], e, big);
                    loc = add2(loc, x[i]);
                }
                float S = tm.sum(fmaf(big, 0.0f, loc.x + loc.y));      // NaN where `big` is infinite
                if (!(S >= kBalTinySum)) {
                    float y[NE], m = -INFINITY, sum = 0.0f, slope;
                    bal_load<NV, VEC>(a.logits + static_cast<size_t>(t) * a.E, a.E, tm.wt, lane, -INFINITY, y);
#pragma unroll
                    for (int i = 0; i < NE; ++i) m = fmaxf(m, y[i]);
                    m = tm.max(m);
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        y[i] = sigmoid_over(y[i], m, slope);
                        sum += y[i];
                    }
                    S = tm.sum(sum);
#pragma unroll
                    for (int i = 0; i < NE / 2; ++i) x[i] = make_float2(y[2 * i], y[2 * i + 1]);
                }
                const float inv = S == 0.0f ? 0.0f : rcp_approx(S);
#pragma unroll
                for (int i = 0; i < NE / 2; ++i) acc[i] = fma2(x[i], make_float2(inv, inv), acc[i]);
                if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
                ++n;
            }
            id = id1, id1 = id2;
        }
#pragma unroll
        for (int i = 0; i < NE / 2; ++i) {
            const int e0 = bal_expert<NV, VEC>(tm.wt, lane, 2 * i), e1 = bal_expert<NV, VEC>(tm.wt, lane, 2 * i + 1);
            if (e0 < a.E) sums[team * a.E + e0] = acc[i].x;
            if (e1 < a.E) sums[team * a.E + e1] = acc[i].y;
        }
        if (tm.wt == 0 && lane == 0 && n) atomicAdd(&s_n, n);
        __syncthreads();
        const size_t slot = CL ? static_cast<size_t>(q) : static_cast<size_t>(blockIdx.x) + q;
        float* dst_p = (CL ? own_p : a.slot_p) + slot * a.E;
        int32_t* dst_c = (CL ? own_c : a.slot_c) + slot * a.E;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float p = sums[e];
            for (int m = 1; m < a.teams; ++m) p += sums[m * a.E + e];
            dst_p[e] = p;
            dst_c[e] = hist[e];
            hist[e] = 0;
        }
        if (threadIdx.x == 0) {
            (CL ? own_n : a.slot_n)[slot] = s_n;
            s_n = 0;
        }
        __syncthreads();
    }
    feed.drain();
    if constexpr (CL) {
        __shared__ float s_dot[kWarps];
        const int rank = blockIdx.x, ranks = gridDim.x;
        cluster_sync_all();
        for (int q = rank; q < a.Q; q += ranks) {
            int n = 0;
            for (int r = 0; r < ranks; ++r) n += __float_as_int(ld_cluster_f32(reinterpret_cast<const float*>(own_n + q), r));
            float dot = 0.0f;
            for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
                float p = 0.0f;
                int c = 0;
#pragma unroll
                for (int r = 0; r < kBalCluster; ++r) {
                    p += ld_cluster_f32(own_p + q * a.E + e, r);
                    c += __float_as_int(ld_cluster_f32(reinterpret_cast<const float*>(own_c + q * a.E + e), r));
                }
                a.prob_sums[static_cast<size_t>(q) * a.E + e] = p;
                a.counts[static_cast<size_t>(q) * a.E + e] = c;
                dot += static_cast<float>(c) * p;
            }
            dot = warp_tree_sum(n > 0 ? dot : 0.0f);
            if (lane == 0) s_dot[warp] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < static_cast<int>(blockDim.x) / 32; ++w) dot += s_dot[w];
                const float fn = static_cast<float>(n);
                st_cluster(own_l + q, 0, n > 0 ? dot * (static_cast<float>(a.E) / static_cast<float>(a.k)) / fn / fn : 0.0f);
                st_cluster(reinterpret_cast<float*>(own_n) + a.Q * 2 + q, 0, __int_as_float(n > 0));
                a.seq_tokens[q] = n;
            }
            __syncthreads();
        }
        cluster_sync_all();      // also keeps every CTA's shared memory until its readers are done
        if (rank == 0 && threadIdx.x == 0) {
            double l = 0.0;
            int some = 0;
            for (int q = 0; q < a.Q; ++q) l += own_l[q], some += own_n[2 * a.Q + q];
            a.loss[0] = static_cast<float>(l * a.coeff / (some > 0 ? some : 1));
        }
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

template <bool MAX, int M>
__device__ __forceinline__ void group_join(float (&v)[M], int G) {      // each over the G lanes of a row
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        if (off >= 8 && off >= G) break;      // G is 8, 16 or 32
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const float o = __shfl_xor_sync(0xffffffffu, v[j], off);
            v[j] = MAX ? fmaxf(v[j], o) : v[j] + o;
        }
    }
}

// The gate's own gradient for M times the picks of 32 / G rows, G lanes a
// row (G a power of two >= k): this lane's picks `id` (-1: none) with logits xj
// and incoming gradients dw.  The rows are independent, so their chains of sums
// run side by side.  `tags`: two times kBalTags bytes a row of the warp's own
// shared memory, any contents.
template <int M>
__device__ __forceinline__ void gate_pick_grad(const int (&id)[M], const float (&xj)[M],
                                               const float (&dw)[M], int G, volatile uint8_t* tags,
                                               float (&d)[M]) {
    const int lane = threadIdx.x & 31;
    float s[M], om[M], tot[M];
    int tiny = 0, twice = 0;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        // Two picks of one expert find each other's mark; so may two of 1024 experts apart, which the match below
        // tells from them (a match costs about 1000 cycles for 32 different values).  The marks alternate between
        // two areas, so one is written while the other may still be read.
        volatile uint8_t* tag = tags + (((j & 1) * 32 + lane) / G * kBalTags) + (id[j] & (kBalTags - 1));
        if (id[j] >= 0) *tag = static_cast<uint8_t>(lane);
        __syncwarp();
        twice |= id[j] >= 0 ? *tag ^ lane : 0;
    }
#pragma unroll
    for (int j = 0; j < M; ++j) {
        const float u = ex2_approx(fabsf(xj[j]) * -kLog2e), r = rcp_approx(1.0f + u);
        om[j] = xj[j] >= 0.0f ? u * r : r;
        s[j] = id[j] < 0 ? 0.0f : xj[j] >= 0.0f ? r : u * r;
        tot[j] = s[j];
    }
    group_join<false, M>(tot, G);
#pragma unroll
    for (int j = 0; j < M; ++j) tiny |= id[j] >= 0 && !(tot[j] >= kBalTinySum) ? 1 : 0;
    if (__any_sync(0xffffffffu, tiny != 0)) {      // relative to the row's largest, as in the loss
        float m[M], slope;
#pragma unroll
        for (int j = 0; j < M; ++j) m[j] = id[j] >= 0 ? xj[j] : -INFINITY;
        group_join<true, M>(m, G);
#pragma unroll
        for (int j = 0; j < M; ++j) {
            s[j] = id[j] < 0 ? 0.0f : sigmoid_over(xj[j], m[j], slope);
            tot[j] = s[j];
        }
        group_join<false, M>(tot, G);
    }
    float dot[M];
#pragma unroll
    for (int j = 0; j < M; ++j) {
        // divided: a token's only pick has the weight 1 and no gradient
        s[j] = tot[j] == 0.0f ? 0.0f : __fdiv_rn(s[j], tot[j]);
        dot[j] = id[j] < 0 ? 0.0f : dw[j] * s[j];
    }
    group_join<false, M>(dot, G);
#pragma unroll
    for (int j = 0; j < M; ++j) d[j] = s[j] * om[j] * (dw[j] - dot[j]);
    if (__any_sync(0xffffffffu, twice != 0)) {   // the same expert twice in a row: added in slot order
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const unsigned same = __match_any_sync(0xffffffffu, id[j] < 0 ? -1 - lane : id[j] | (lane / G) << 16);
            float z = 0.0f;
#pragma unroll 1
            for (int i = 0; i < 32; ++i) {
                const float di = __shfl_sync(0xffffffffu, d[j], i);
                if (same >> i & 1u) z += di;
            }
            d[j] = z;
        }
    }
}

// A gate warp's whole work: the lists of teams g, g + kBalGateWarps, ... (M of
// them at most), side by side.  All loads go to valid places whether their values
// count or not, and are looked at a turn later, so none is branched around or
// waited for where it starts.
template <int M>
__device__ __forceinline__ void gate_lists(const BalArgs& a, int g, int t0, int t1, volatile uint8_t* tags,
                                        int2 (*list)[kBalLists][32], uint64_t (*list_full)[kBalLists],
                                        uint64_t (*list_empty)[kBalLists]) {
    const int lane = threadIdx.x & 31;
    const int G = bal_group(a.k), batch = 32 / G;
    int lists[M];            // of each team
#pragma unroll
    for (int j = 0; j < M; ++j) {
        const int team = g + j * kBalGateWarps;
        const int rows = team < a.teams && t0 + team < t1 ? (t1 - t0 - team + a.teams - 1) / a.teams : 0;
        lists[j] = (rows + batch - 1) / batch;
    }
    if (lists[0] == 0) return;
    // this lane's token of list b and team g is first + b * step, those of the other teams kBalGateWarps further each
    const int64_t first = t0 + g + static_cast<int64_t>(lane / G) * a.teams, step = static_cast<int64_t>(batch) * a.teams;
    const int pick = min(lane % G, a.k - 1);
    const uint32_t experts = lane % G < a.k ? static_cast<uint32_t>(a.E) : 0u;
    int64_t tp = first, tv = first;         // token of the next fetch of picks and of values
    auto fetch_picks = [&](int (&d)[M], int (&m)[M]) {
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const int64_t t = min(tp + j * kBalGateWarps, static_cast<int64_t>(t1 - 1));
            d[j] = a.ids[t * a.k + pick];
            m[j] = a.mask[t];
        }
        tp += step;
    };
    auto fetch_values = [&](int (&d)[M], const int (&m)[M], float (&x)[M], float (&w)[M]) {
#pragma unroll
        for (int j = 0; j < M; ++j) {
            const int64_t t = min(tv + j * kBalGateWarps, static_cast<int64_t>(t1 - 1));
            uint32_t below = tv + j * kBalGateWarps < t1 ? experts : 0u;      // ids that count are below it
            below = m[j] != 0 ? below : 0u;
            d[j] = static_cast<uint32_t>(d[j]) < below ? d[j] : -1;
            x[j] = a.logits[t * a.E + max(d[j], 0)];
            w[j] = a.grad_w[t * a.k + pick];
        }
        tv += step;
    };
    int id[M], id1[M], m1[M];
    float xj[M], dw[M];
    fetch_picks(id, m1);
    fetch_values(id, m1, xj, dw);
    fetch_picks(id1, m1);
    int my_team = g, my_lists = 0;          // lanes 0 .. M - 1 see to a team each
#pragma unroll
    for (int j = 0; j < M; ++j)
        if (lane == j) my_team = g + j * kBalGateWarps, my_lists = lists[j];
    bool dead = false;
    int slot = 0, phase = 1;
    for (int b = 0; b < lists[0]; ++b) {
        int id2[M], m2[M];
        float xj1[M], dw1[M], d[M];
        fetch_picks(id2, m2);
        fetch_values(id1, m1, xj1, dw1);
        gate_pick_grad(id, xj, dw, G, tags, d);
        if (b >= kBalLists && b < my_lists && !dead)      // a team takes every list that is made for it
            dead = !mbar_wait_bounded(&list_empty[my_team][slot], static_cast<uint32_t>(phase), kBalTimeout);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (b < lists[j]) list[g + j * kBalGateWarps][slot][lane] = make_int2(id[j], __float_as_int(d[j]));
        __syncwarp();
        if (b < my_lists) mbar_arrive(&list_full[my_team][slot]);
        if (++slot == kBalLists) slot = 0, phase ^= 1;
#pragma unroll
        for (int j = 0; j < M; ++j)
            id[j] = id1[j], id1[j] = id2[j], m1[j] = m2[j], xj[j] = xj1[j], dw[j] = dw1[j];
    }
}

// The gradient of the logits.  A team of warps keeps its row in registers, as in
// the loss.  The gate's own gradient, a chain of dependent sums over few lanes,
// is the work of kBalGateWarps warps beside the teams: each serves every
// kBalGateWarps-th team and leaves the entries (expert, gradient) of 32 / G rows
// at a time in the team's ring of lists.  A warp of the team lays the entries
// that fall to its part of the row into a part-row of shared memory (zero
// elsewhere) and adds that in the dense pass, so every logit's gradient is
// written once, in full lines.  (With the gate in the teams themselves 32768 x
// 2560 took 177 us instead of 133.)
template <int NV, bool VEC, bool BAL>
__global__ void __launch_bounds__((kBalGradWarps + kBalGateWarps) * 32, 1) gate_grad_kernel(const BalArgs a) {
    constexpr int NE = 4 * NV;
    extern __shared__ __align__(128) uint8_t bal_smem[];
    __shared__ float2 red[kBalGradWarps][2 * kBalMaxTeam];
    __shared__ __align__(8) uint64_t bars[kBalGradWarps * kBalRing];
    __shared__ __align__(8) uint64_t list_full[kBalGradWarps][kBalLists], list_empty[kBalGradWarps][kBalLists];
    __shared__ int2 list[kBalGradWarps][kBalLists][32];
    __shared__ int s_some;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int teams_warps = a.W * a.teams;
    float* adds = reinterpret_cast<float*>(bal_smem + (BAL ? bal_ring_bytes<NV>(teams_warps, a.ring) : 0));
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
    const int t0 = static_cast<int>(min(c0, static_cast<int64_t>(a.T)));
    const int t1 = static_cast<int>(min(c0 + a.tokens, static_cast<int64_t>(a.T)));
    for (int e = threadIdx.x; e < teams_warps * NV * 128; e += blockDim.x) adds[e] = 0.0f;
    for (int i = threadIdx.x; i < kBalGradWarps * kBalRing; i += blockDim.x) mbar_init(&bars[i], 1);
    for (int i = threadIdx.x; i < kBalGradWarps * kBalLists; i += blockDim.x) {
        mbar_init(&list_full[i / kBalLists][i % kBalLists], 1);
        mbar_init(&list_empty[i / kBalLists][i % kBalLists], a.W);
    }
    if (threadIdx.x == 0) s_some = 0;
    fence_mbar_init();
    __syncthreads();
    griddep_wait();
    griddep_launch();
    const int G = bal_group(a.k), batch = 32 / G;
    float unit = 0.0f;
    if constexpr (BAL) {
        int some = 0;
        for (int q = threadIdx.x; q < a.Q; q += blockDim.x) some += a.seq_tokens_in[q] > 0;
        if (some) atomicAdd(&s_some, some);
        __syncthreads();
        unit = a.grad_loss[0] * a.coeff * (static_cast<float>(a.E) / static_cast<float>(a.k)) /
               static_cast<float>(s_some > 0 ? s_some : 1);
    }

    if (warp >= teams_warps) {
        const int g = warp - teams_warps;
        volatile uint8_t* tags = reinterpret_cast<uint8_t*>(adds + teams_warps * NV * 128) + g * 2 * batch * kBalTags;
        if (a.teams > 2 * kBalGateWarps)
            gate_lists<4>(a, g, t0, t1, tags, list, list_full, list_empty);
        else if (a.teams > kBalGateWarps)
            gate_lists<2>(a, g, t0, t1, tags, list, list_full, list_empty);
        else
            gate_lists<1>(a, g, t0, t1, tags, list, list_full, list_empty);
        return;
    }

    const int team = warp / a.W;
    Team tm{red[team], a.W, 1 + team, warp % a.W, lane, 0};
    float* add = adds + static_cast<size_t>(warp) * NV * 128;      // this warp's part of a row
    RowFeed<NV, VEC> feed;
    RowMask mask;
    mask.start(a, lane, t0 + team, t1);
    if constexpr (BAL) feed.start(a, tm, warp, t0 + team, t1, bal_smem, bars);
    const bool gate = a.grad_w != nullptr;
    bool dead = false;
    int q = BAL ? first_sequence(a, t0) : a.Q, q_lo = 0, q_hi = -1;
    float2 g[NE / 2];
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) g[i] = make_float2(0.0f, 0.0f);
    int slot = 0, phase = 0, in_batch = 0;
    float* out = a.grad + static_cast<size_t>(t0 + team < t1 ? t0 + team : 0) * a.E;
    for (int t = t0 + team; t < t1; t += a.teams, out += static_cast<size_t>(a.teams) * a.E) {
        const bool valid = mask.next();
        bool in_seq = false;
        float2 x[NE / 2];
        if constexpr (BAL) {
            feed.take(x);
            if (t >= q_hi) {
                while (q < a.Q && (q_hi = clamp_offset(a, q + 1)) <= t) ++q;
                if (q >= a.Q) q_hi = a.T;
                q_lo = q < a.Q ? clamp_offset(a, q) : a.T;
                const int n = q < a.Q ? a.seq_tokens_in[q] : 0;
                const float fn = static_cast<float>(n);
                const float c = n > 0 ? unit / fn / fn : 0.0f;
                const int32_t* row_c = a.counts_in + static_cast<size_t>(q < a.Q ? q : 0) * a.E;
#pragma unroll
                for (int i = 0; i < NE / 2; ++i) {
                    const int e0 = bal_expert<NV, VEC>(tm.wt, lane, 2 * i), e1 = bal_expert<NV, VEC>(tm.wt, lane, 2 * i + 1);
                    g[i].x = e0 < a.E ? c * static_cast<float>(row_c[e0]) : 0.0f;
                    g[i].y = e1 < a.E ? c * static_cast<float>(row_c[e1]) : 0.0f;
                }
            }
            in_seq = valid && t >= q_lo;
        }
        // this row's entries that fall to this warp
        int at = -1;
        if (gate) {
            if (in_batch == 0 && !dead)
                dead = !mbar_wait_bounded(&list_full[team][slot], static_cast<uint32_t>(phase), kBalTimeout);
            int2 entry = make_int2(-1, 0);
            if (lane < G) entry = list[team][slot][in_batch * G + lane];
            __syncwarp();       // also: behind the lanes that cleared the last row's entries
            if (++in_batch == batch) {
                in_batch = 0;
                if (lane == 0) mbar_arrive(&list_empty[team][slot]);
                if (++slot == kBalLists) slot = 0, phase ^= 1;
            }
            at = entry.x - tm.wt * NV * 128;
            if (entry.x < 0 || at >= NV * 128) at = -1;
            if (at >= 0) add[at] = __int_as_float(entry.y);
            __syncwarp();
        }
        float2 S2 = make_float2(0.0f, 0.0f), G2 = S2;
        const bool dense = BAL && in_seq;
        if (dense) {
            float2 sum = make_float2(0.0f, 0.0f), dot = sum;
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < NE / 2; ++i) {
                float2 e;
                const float2 s = sigmoid2(x[i], e, big);
                x[i] = mul2(mul2(e, s), s);         // s (1 - s) = exp(-x) s^2
                sum = add2(sum, s);
                dot = fma2(g[i], s, dot);
            }
            float2 all = tm.sum(make_float2(fmaf(big, 0.0f, sum.x + sum.y), dot.x + dot.y));
            if (!(all.x >= kBalTinySum)) {
                float y[NE], m = -INFINITY;
                bal_load<NV, VEC>(a.logits + static_cast<size_t>(t) * a.E, a.E, tm.wt, lane, -INFINITY, y);
#pragma unroll
                for (int i = 0; i < NE; ++i) m = fmaxf(m, y[i]);
                m = tm.max(m);
                all = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    float slope;
                    const float s = sigmoid_over(y[i], m, slope);
                    all.x += s;
                    all.y = fmaf(i % 2 ? g[i / 2].y : g[i / 2].x, s, all.y);
                    (i % 2 ? x[i / 2].y : x[i / 2].x) = slope;
                }
                all = tm.sum(all);
            }
            const float S = all.x == 0.0f ? 0.0f : __frcp_rn(all.x);
            const float G1 = all.y * S;
            S2 = make_float2(S, S), G2 = make_float2(-G1, -G1);
        } else {
#pragma unroll
            for (int i = 0; i < NE / 2; ++i) x[i] = make_float2(0.0f, 0.0f);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const float2 lo = mul2(x[2 * v], S2), hi = mul2(x[2 * v + 1], S2);
            // a row without a part in the loss takes none of its g, which may be infinite or NaN
            const float2 none = make_float2(0.0f, 0.0f);
            const float2 gl = dense ? add2(g[2 * v], G2) : none, gh = dense ? add2(g[2 * v + 1], G2) : none;
            if constexpr (VEC) {
                const int e = bal_expert<NV, VEC>(tm.wt, lane, 4 * v);
                if (e < a.E) {
                    const float4 z = *reinterpret_cast<const float4*>(add + 128 * v + 4 * lane);
                    const float2 p = fma2(lo, gl, make_float2(z.x, z.y)), r = fma2(hi, gh, make_float2(z.z, z.w));
                    __stcs(reinterpret_cast<float4*>(out + e), make_float4(p.x, p.y, r.x, r.y));
                }
            } else {
                const float w[4] = {lo.x * gl.x, lo.y * gl.y, hi.x * gh.x, hi.y * gh.y};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = bal_expert<NV, VEC>(tm.wt, lane, 4 * v + i);
                    if (e < a.E) __stcs(out + e, w[i] + add[(4 * v + i) * 32 + lane]);
                }
            }
        }
        __syncwarp();
        if (at >= 0) add[at] = 0.0f;
    }
    if constexpr (BAL) feed.drain();
}

template <typename F>
cudaError_t bal_launch(F* kernel, int ctas, int threads, size_t smem, int cluster, const BalArgs& a, cudaStream_t s) {
    if (smem > 24 * 1024) {      // with the kernel's static shared memory above the 48 KB of an unset limit
        const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int NV, bool VEC>
cudaError_t launch_balance_nv(const BalPlan& p, const BalArgs& a, cudaStream_t s) {
    const int warps = p.W * p.teams;
    size_t smem = bal_ring_bytes<NV>(warps, p.ring) + static_cast<size_t>(p.teams + 1) * a.E * 4;
    if (!p.cluster) return bal_launch(balance_kernel<NV, VEC, false>, p.ctas, warps * 32, smem, 1, a, s);
    smem += static_cast<size_t>(a.Q) * (2 * a.E + 3) * 4;
    return bal_launch(balance_kernel<NV, VEC, true>, kBalCluster, warps * 32, smem, kBalCluster, a, s);
}
template <bool VEC>
cudaError_t launch_balance_main(const BalPlan& p, const BalArgs& a, cudaStream_t s) {
    switch (p.nv) {
        case 1: return launch_balance_nv<1, VEC>(p, a, s);
        case 2: return launch_balance_nv<2, VEC>(p, a, s);
        case 3: return launch_balance_nv<3, VEC>(p, a, s);
        default: return launch_balance_nv<4, VEC>(p, a, s);
    }
}
template <int NV, bool VEC, bool BAL>
cudaError_t launch_gate_grad_nv(const BalPlan& p, const BalArgs& a, cudaStream_t s) {
    const int warps = p.W * p.teams, gate = a.grad_w != nullptr ? kBalGateWarps : 0;
    const size_t smem = (BAL ? bal_ring_bytes<NV>(warps, p.ring) : 0) + static_cast<size_t>(warps) * NV * 512 +
                        static_cast<size_t>(gate) * 2 * (32 / bal_group(a.k)) * kBalTags;
    return bal_launch(gate_grad_kernel<NV, VEC, BAL>, p.ctas, (warps + gate) * 32, smem, 1, a, s);
}
template <bool VEC, bool BAL>
cudaError_t launch_gate_grad(const BalPlan& p, const BalArgs& a, cudaStream_t s) {
    switch (p.nv) {
        case 1: return launch_gate_grad_nv<1, VEC, BAL>(p, a, s);
        case 2: return launch_gate_grad_nv<2, VEC, BAL>(p, a, s);
        case 3: return launch_gate_grad_nv<3, VEC, BAL>(p, a, s);
        default: return launch_gate_grad_nv<4, VEC, BAL>(p, a, s);
    }
}

size_t pad16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }
int bal_parts(int E) { return (E + kFinExperts - 1) / kFinExperts; }

}  // namespace

size_t balance_workspace_bytes(int T, int E, int Q) {
    const BalPlan p = bal_plan(T, E, Q, false);
    if (p.cluster) return 0;
    const size_t slots = static_cast<size_t>(p.ctas) + Q;
    return 16 + 2 * pad16(slots * E * 4) + pad16(slots * 4) + pad16(static_cast<size_t>(Q) * bal_parts(E) * 4);
}

cudaError_t launch_balance_loss(const BalanceLaunch& b, cudaStream_t s) {
    const BalPlan p = bal_plan(b.T, b.E, b.Q, false);
    BalArgs a{};
    a.logits = b.logits, a.ids = b.ids, a.mask = b.mask, a.offsets = b.offsets;
    a.T = b.T, a.E = b.E, a.k = b.k, a.Q = b.Q, a.coeff = b.coeff;
    a.W = p.W, a.teams = p.teams, a.tokens = p.tokens, a.ring = p.ring;
    a.loss = b.loss, a.counts = b.counts, a.prob_sums = b.prob_sums, a.seq_tokens = b.seq_tokens;
    if (!p.cluster) {
        const size_t slots = static_cast<size_t>(p.ctas) + b.Q;
        uint8_t* w = static_cast<uint8_t*>(b.workspace);
        a.ticket = reinterpret_cast<unsigned int*>(w);
        a.slot_p = reinterpret_cast<float*>(w += 16);
        a.slot_c = reinterpret_cast<int32_t*>(w += pad16(slots * b.E * 4));
        a.slot_n = reinterpret_cast<int32_t*>(w += pad16(slots * b.E * 4));
        a.loss_part = reinterpret_cast<float*>(w += pad16(slots * 4));
    }
    const cudaError_t e = b.E % 4 == 0 ? launch_balance_main<true>(p, a, s) : launch_balance_main<false>(p, a, s);
    if (e != cudaSuccess || p.cluster) return e;
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
    const BalPlan p = bal_plan(b.T, b.E, b.Q, true);
    BalArgs a{};
    a.logits = b.logits, a.ids = b.ids, a.mask = b.mask, a.offsets = b.offsets;
    a.T = b.T, a.E = b.E, a.k = b.k, a.Q = b.Q, a.coeff = b.coeff;
    a.W = p.W, a.teams = p.teams, a.tokens = p.tokens, a.ring = p.ring;
    a.grad_w = b.grad_w, a.grad_loss = b.grad_loss, a.counts_in = b.counts, a.seq_tokens_in = b.seq_tokens;
    a.grad = b.grad;
    const bool bal = b.grad_loss != nullptr;
    if (b.E % 4 == 0) return bal ? launch_gate_grad<true, true>(p, a, s) : launch_gate_grad<true, false>(p, a, s);
    return bal ? launch_gate_grad<false, true>(p, a, s) : launch_gate_grad<false, false>(p, a, s);
}

}  // namespace mb
