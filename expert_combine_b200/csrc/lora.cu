// lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t, :] = base[t, :] + scale_a * (x[t, :] A_a^T) B_a^T,  a = adapter_ids[t]
// with x [T, H], A [L, R, H], B [L, N, R] in BF16 and base/out [T, N] in FP32
// or BF16; a token whose id is outside [0, L) keeps its row of base.
//
// Two products of very different shape: the first ("shrink") reads x and A,
// reduces over H and leaves v [T, R] in FP32; the second ("expand") reads v
// and B, and adds to base over N.  R is small, so both are bound by their
// reads and writes, and by latency when there are few tokens.
//
// Few tokens (decode).  One launch, a cluster of 8 CTAs for each token.  Tokens
// of one adapter are taken in groups of up to 8 (the N of an m16n8k16 MMA, the
// adapter's 16 ranks its M): the cluster of token t works on the group that t
// leads, i.e. whose earlier tokens of the same adapter number a multiple of 8,
// and the clusters of the other tokens leave at once.  Every CTA finds that out
// for itself from the ids (one ballot per warp), so nothing is sorted
// beforehand.  The CTAs of a cluster split H: operands come straight from memory
// into the MMA's registers.  Which k a lane's registers stand for is free as
// long as A and x agree, so a lane takes 8 consecutive k of its row as one
// 16-byte load, and two MMAs use up the four words of each.  Then every CTA
// reads the eight partial v through distributed shared memory, adds them in
// order and forms its share of the columns with FP32 multiply-adds, two columns
// a thread.  B is asked into L2 before the first product begins.
//
// Many tokens (prefill).  The tokens are sorted by adapter (a one-CTA kernel, or
// the dispatch of the routing entries for the larger batches: one "pick" a
// token, L "experts"), each adapter's run is cut into tiles of 128 tokens, and
// both products run on the tensor cores (tcgen05, accumulators in tensor
// memory), one persistent CTA per SM: a TMA thread, an MMA thread, four loading
// and eight epilogue warps.
//   shrink  All tiles' steps of 128 k form one line that is cut into equal
//     pieces, one per CTA, so the SMs finish together whatever the sizes of
//     the groups.  The rows of a tile lie anywhere in x: four warps fetch them
//     in 16-byte pieces.  A tile that several CTAs share is summed by the one
//     that arrives last, from the partials, in the CTAs' order (an integer
//     counter per tile; the sum's order does not depend on the arrival).  It
//     writes v scaled and split into BF16 parts (3 for FP32 outputs: v whole; 2 for
//     BF16 outputs: 2^-16 of v is left), in the layout of the next MMA's operand.
//   expand  Work items are a tile x 128 columns, cut the same way.  D = sum over
//     the parts v_p B^T; base arrives in the swizzled layout in which an epilogue
//     thread reads its row without bank conflicts, the sum replaces it there,
//     and the warp writes whole 128-byte rows of out.
// In steady state both move about 25 bytes a cycle and SM between L2 and the
// SMs.  From a graph, 8192 tokens x 8192 -> 8192, rank 64, BF16: 94 us (x, base
// and out alone are 61 at the copy rate; called one by one 96 to 101); -> 256
// columns, rank 32, FP32: 47 us.
#include "internal.h"
#include "common.cuh"
#include "tmap.h"
#include "mma.cuh"

namespace mb {

namespace {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraTokens = 256;           // most tokens of this path,
constexpr int kLoraTokensWide = 192;       // and of more than kLoraNarrow ranks, see lora_few
constexpr int kLoraNarrow = 32;
constexpr int kLoraGroup = 8;              // tokens per group
constexpr int kLoraCluster = 8;            // CTAs per group

struct LoraArgs {
    const uint16_t* x;        // [T, H]
    const uint16_t* a;        // [L, R, H]
    const uint16_t* b;        // [L, N, R]
    const int32_t* ids;       // [T]
    const float* scales;      // [L] or NULL
    const void* base;         // [T, N]
    void* out;                // [T, N]
    int T, H, N, R, L;
    int kc;                   // H is cut into runs of kc, one per CTA of a cluster
    int nc;                   // and N into runs of nc
};

// The group that token t leads: its members in order (s_member) and their
// number, or 0 when t leads none; *id is t's adapter, -1 for none.
__device__ __forceinline__ int lora_group(const LoraArgs& a, int t, int* id, uint32_t* s_mask, int* s_member) {
    const int mine = threadIdx.x < a.T ? a.ids[threadIdx.x] : -1, my = a.ids[t];
    *id = my >= 0 && my < a.L ? my : -1;
    if (*id < 0) return 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t same = __ballot_sync(0xffffffffu, mine == my);
    if (lane == 0) s_mask[warp] = same;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < (t >> 5); ++w) before += __popc(s_mask[w]);
    before += __popc(s_mask[t >> 5] & ((1u << (t & 31)) - 1u));
    if (before % kLoraGroup != 0) return 0;
    // token threadIdx.x is the group's member number (tokens of the adapter between t and it)
    int rank = -before;
    for (int w = 0; w < warp; ++w) rank += __popc(s_mask[w]);
    rank += __popc(same & ((1u << lane) - 1u));
    if (mine == my && rank >= 0 && rank < kLoraGroup) s_member[rank] = threadIdx.x;
    int all = -before;
    for (int w = 0; w < kLoraWarps; ++w) all += __popc(s_mask[w]);
    __syncthreads();
    return all < kLoraGroup ? all : kLoraGroup;
}

__device__ __forceinline__ void mma_16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename O>
__device__ __forceinline__ float2 load2(const void* p, size_t i);
template <>
__device__ __forceinline__ float2 load2<float>(const void* p, size_t i) {
    return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
}
template <>
__device__ __forceinline__ float2 load2<uint16_t>(const void* p, size_t i) {
    return unpack_bf16x2(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i));
}
template <typename O>
__device__ __forceinline__ void store2(void* p, size_t i, float2 v);
template <>
__device__ __forceinline__ void store2<float>(void* p, size_t i, float2 v) {
    *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = v;
}
template <>
__device__ __forceinline__ void store2<uint16_t>(void* p, size_t i, float2 v) {
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + i) = pack_bf16x2_rn(v);
}

// Two columns of G tokens: base + v B^T, v [G][R] in shared memory.
template <int G, typename O>
__device__ __forceinline__ void lora_columns(const LoraArgs& a, const float* v, const int* member, int n,
                                             const uint16_t* b, int col) {
    float2 base[G], acc[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
        base[j] = j < n ? load2<O>(a.base, static_cast<size_t>(member[j]) * a.N + col) : make_float2(0.0f, 0.0f);
        acc[j] = make_float2(0.0f, 0.0f);
    }
#pragma unroll 2
    for (int r = 0; r < a.R; r += 8) {
        const uint4 b0 = ld_nc_v4(b + r), b1 = ld_nc_v4(b + a.R + r);
        const uint32_t w0[4] = {b0.x, b0.y, b0.z, b0.w}, w1[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 p0 = unpack_bf16x2(w0[2 * h]), q0 = unpack_bf16x2(w0[2 * h + 1]);
            const float2 p1 = unpack_bf16x2(w1[2 * h]), q1 = unpack_bf16x2(w1[2 * h + 1]);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float4 f = *reinterpret_cast<const float4*>(v + j * a.R + r + 4 * h);
                acc[j] = fma2(make_float2(f.x, f.x), make_float2(p0.x, p1.x), acc[j]);
                acc[j] = fma2(make_float2(f.y, f.y), make_float2(p0.y, p1.y), acc[j]);
                acc[j] = fma2(make_float2(f.z, f.z), make_float2(q0.x, q1.x), acc[j]);
                acc[j] = fma2(make_float2(f.w, f.w), make_float2(q0.y, q1.y), acc[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < G; ++j)
        if (j < n) store2<O>(a.out, static_cast<size_t>(member[j]) * a.N + col, add2(base[j], acc[j]));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// MT tiles of 16 ranks.  Three CTAs to an SM, as far as few ranks allow: 128
// tokens over 32 adapters take 11.5 us against 13.3 with the two that the
// unbounded registers leave (one token 3.9 against 3.8).
template <int MT, typename O>
__global__ void __launch_bounds__(kLoraThreads, MT <= 2 ? 3 : 1) lora_few_kernel(const LoraArgs a) {
    __shared__ uint32_t s_mask[kLoraWarps];
    __shared__ int s_member[kLoraGroup];
    __shared__ __align__(16) float s_w[kLoraWarps][kLoraGroup][MT * 16];   // the warps' sums
    __shared__ __align__(16) float s_part[kLoraGroup * MT * 16];           // the CTA's: [token][rank]
    __shared__ __align__(16) float s_v[kLoraGroup * MT * 16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x / kLoraCluster, part = blockIdx.x % kLoraCluster;
    griddep_wait();
    griddep_launch();
    const int n0 = part * a.nc, n1 = min(a.N, n0 + a.nc);
    int id;
    const int n = lora_group(a, t, &id, s_mask, s_member);
    if (n == 0) {       // the whole cluster leaves
        if (id < 0 && a.out != a.base)
            for (int col = n0 + 2 * threadIdx.x; col < n1; col += 2 * kLoraThreads)
                store2<O>(a.out, static_cast<size_t>(t) * a.N + col, load2<O>(a.base, static_cast<size_t>(t) * a.N + col));
        return;
    }
    {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(a.b + (static_cast<size_t>(id) * a.N + n0) * a.R);
        for (int i = threadIdx.x * 128; i < (n1 - n0) * a.R * 2; i += kLoraThreads * 128) prefetch_l2(b + i);
    }

    const int g = lane >> 2, c = lane & 3;
    const int k_end = min((part + 1) * a.kc, a.H);
    const int tok = g < n ? s_member[g] : -1;
    const uint16_t* xr = a.x + static_cast<size_t>(tok < 0 ? 0 : tok) * a.H;
    const uint16_t* ar = a.a + (static_cast<size_t>(id) * a.R + g) * a.H;
    float acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
    for (int k = part * a.kc + warp * 32 + c * 8; k - c * 8 < k_end; k += kLoraWarps * 32) {
        const bool in = k < k_end;
        const uint4 xv = in && tok >= 0 ? ld_nc_v4(xr + k) : zero;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint4 lo = in && 16 * m + g < a.R ? ld_nc_v4(ar + static_cast<size_t>(16 * m) * a.H + k) : zero;
            const uint4 hi =
                in && 16 * m + g + 8 < a.R ? ld_nc_v4(ar + static_cast<size_t>(16 * m + 8) * a.H + k) : zero;
            mma_16n8k16(acc[m], lo.x, hi.x, lo.y, hi.y, xv.x, xv.y);
            mma_16n8k16(acc[m], lo.z, hi.z, lo.w, hi.w, xv.z, xv.w);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        s_w[warp][2 * c][16 * m + g] = acc[m][0];
        s_w[warp][2 * c + 1][16 * m + g] = acc[m][1];
        s_w[warp][2 * c][16 * m + g + 8] = acc[m][2];
        s_w[warp][2 * c + 1][16 * m + g + 8] = acc[m][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kLoraGroup * MT * 16; i += kLoraThreads) {
        float v = (&s_w[0][0][0])[i];
#pragma unroll
        for (int w = 1; w < kLoraWarps; ++w) v += (&s_w[w][0][0])[i];
        s_part[i] = v;
    }
    cluster_sync_all();
    const float scale = a.scales != nullptr ? a.scales[id] : 1.0f;
    for (int i = threadIdx.x; i < n * a.R; i += kLoraThreads) {
        const int j = i / a.R, r = i - j * a.R;
        float p[kLoraCluster], v = 0.0f;
#pragma unroll
        for (int q = 0; q < kLoraCluster; ++q) p[q] = ld_cluster_f32(s_part + j * MT * 16 + r, q);
#pragma unroll
        for (int q = 0; q < kLoraCluster; ++q) v += p[q];
        s_v[i] = v * scale;
    }
    __syncthreads();
    for (int col = n0 + 2 * threadIdx.x; col < n1; col += 2 * kLoraThreads) {
        const uint16_t* b = a.b + (static_cast<size_t>(id) * a.N + col) * a.R;
        if (n == 1)
            lora_columns<1, O>(a, s_v, s_member, n, b, col);
        else if (n <= 4)
            lora_columns<4, O>(a, s_v, s_member, n, b, col);
        else
            lora_columns<kLoraGroup, O>(a, s_v, s_member, n, b, col);
    }
    cluster_exit_sync();    // the others have read this CTA's partials
}

template <int MT>
cudaError_t launch_lora_few(const LoraArgs& a, bool bf16, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.T * kLoraCluster);
    cfg.blockDim = dim3(kLoraThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kLoraCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return bf16 ? cudaLaunchKernelEx(&cfg, lora_few_kernel<MT, uint16_t>, a)
                : cudaLaunchKernelEx(&cfg, lora_few_kernel<MT, float>, a);
}

// ------------------------------------------------------------------ many tokens
constexpr int kLmTile = 128;                 // tokens per tile (M of the MMAs)
constexpr int kLmSlab = 64;                  // k per slab: 128 bytes of BF16
constexpr int kLmStep = 2;                   // slabs per ring stage of the shrink kernel
constexpr int kLmSlabBytes = kLmTile * 128;  // 16 KB
constexpr int kLmCols = 128;                 // columns of out per work item
constexpr int kLmThreads = 16 * 32;          // TMA, MMA, 2 warps that copy rows without an adapter, 8 epilogue, 4 loading
constexpr int kLmLoadWarp = 12;              // first of the warps that gather rows
constexpr int kLmCtas = 148;                 // most CTAs of the two kernels; the workspace has a slot for each
constexpr int kLmPlanTokens = 32768;         // most tokens and adapters the one-CTA plan takes
constexpr int kLmPlanAdapters = 1024;
constexpr int kLmEpiWarps = 8;
constexpr int kLmBytes = 208 * 1024;         // ring buffers of a CTA
constexpr int kLmMaxStages = 12;
// Fewest steps worth a CTA of the shrink: the CTA that adds a tile's partials
// waits for each four of them (one adapter, rank 128, 8192 -> 256: 256 tokens
// 33 us with 8 steps, 76 with 1; 512 tokens 33 and 57; 8192 tokens of four
// adapters: the same).
constexpr int kLmLeast = 8;
constexpr int kLmChain = 4;                  // steps (of 2 slabs) the shrink adds up in tensor memory, see below
constexpr unsigned int kLmTimeout = 32u;     // bit 5 of the device status word

struct LmTile {
    int adapter, row0, count, pad;           // rows row0 .. row0 + count - 1 of the grouped order
};

struct LmArgs {
    const int32_t* ids;          // [T]
    const int32_t* offsets;      // [L + 1] first row of each adapter's group (large plans only)
    int32_t* row_token;          // [T] token of a row of the grouped order
    LmTile* tiles;
    int32_t* ntiles;             // [1]
    int32_t* arrived;            // [tiles] CTAs that have left their partial
    float* part;                 // [CTAs + tiles][R][128]
    uint16_t* v;                 // [tiles][parts][ks][128][64]
    const uint16_t* x;
    const float* scales;
    const void* base;
    void* out;
    int T, H, N, R, L;
    int rn;                      // R in steps of 16: columns of the shrink's accumulator
    int ks;                      // 64-wide slabs of R
    int parts;                   // BF16 parts of v
    int stages, b_stages, base_stages, v_bufs;
};

// Tiles of 128 rows of every adapter's group.
__global__ void __launch_bounds__(1024) lora_tiles_kernel(const LmArgs a) {
    __shared__ int s_first[kMaxExperts];     // first tile of each adapter
    __shared__ int s_warp[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = kMaxExperts / 1024;
    griddep_wait();
    griddep_launch();
    int n[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * kPer + j;
        n[j] = e < a.L ? (a.offsets[e + 1] - a.offsets[e] + kLmTile - 1) / kLmTile : 0;
        sum += n[j];
    }
    int scan = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, scan, off);
        if (lane >= off) scan += o;
    }
    if (lane == 31) s_warp[warp] = scan;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    int first = before + scan - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        s_first[tid * kPer + j] = first;
        first += n[j];
    }
    __syncthreads();
    if (tid == 0) *a.ntiles = total;
    for (int i = tid; i < total; i += 1024) a.arrived[i] = 0;
    for (int e = warp; e < a.L; e += 32) {
        const int lo = a.offsets[e], hi = a.offsets[e + 1];
        for (int i = lane; lo + i * kLmTile < hi; i += 32) {
            const int row0 = lo + i * kLmTile;
            a.tiles[s_first[e] + i] = LmTile{e, row0, min(kLmTile, hi - row0), 0};
        }
    }
}

// The whole plan in one CTA: a stable counting sort of the tokens by adapter
// (so the rows' order, and with it every sum's, is the same run to run) and the
// tiles.  Warp w takes the w-th run of tokens 32 at a time; the lanes of one
// adapter find each other by a match, and the warp's running count of that
// adapter gives a token's place among the warp's tokens of the adapter.  The
// general dispatch and the tiles kernel take the larger batches.
__host__ __device__ __forceinline__ size_t lm_plan_bytes(int T, int L) {
    return static_cast<size_t>(2 * ((T + 7) / 8 * 8) + (32 * L + 7) / 8 * 8) * 2 + static_cast<size_t>(2 * (L + 1)) * 4;
}

__global__ void __launch_bounds__(1024) lora_plan_kernel(const LmArgs a) {
    extern __shared__ __align__(16) uint8_t plan_raw[];
    uint16_t* sid = reinterpret_cast<uint16_t*>(plan_raw);      // [T] adapter, 0xffff: none
    uint16_t* place = sid + (a.T + 7) / 8 * 8;                  // [T] among the warp's tokens of the adapter
    uint16_t* cnt = place + (a.T + 7) / 8 * 8;                  // [32][L] the warps' counts, then their first rows
    int* first_row = reinterpret_cast<int*>(cnt + (32 * a.L + 7) / 8 * 8);   // [L + 1]
    int* first_tile = first_row + a.L + 1;                                   // [L + 1]
    __shared__ int2 s_warp[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 32 * a.L; i += 1024) cnt[i] = 0;
    griddep_wait();
    griddep_launch();
#pragma unroll 8
    for (int i = tid; i < a.T; i += 1024) {
        const int id = a.ids[i];
        sid[i] = id >= 0 && id < a.L ? static_cast<uint16_t>(id) : static_cast<uint16_t>(0xffff);
    }
    __syncthreads();
    const int span = (a.T + 1023) / 1024 * 32, lo = warp * span, hi = min(a.T, lo + span);
    uint16_t* mine = cnt + warp * a.L;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane, e = i < hi ? sid[i] : 0xffff;
        const uint32_t same = __match_any_sync(0xffffffffu, e), below = same & ((1u << lane) - 1u);
        const int before = e != 0xffff ? mine[e] : 0;
        __syncwarp();
        if (e != 0xffff) {
            place[i] = static_cast<uint16_t>(before + __popc(below));
            if (below == 0) mine[e] = static_cast<uint16_t>(before + __popc(same));
        }
        __syncwarp();
    }
    __syncthreads();
    // rows and tiles of adapter `tid`, summed over the warps, then over the adapters before it
    const bool some = warp * 32 < a.L;          // this warp has an adapter
    int c[32];
    int2 own = make_int2(0, 0), scan;
    if (some) {
#pragma unroll
        for (int w = 0; w < 32; ++w) c[w] = tid < a.L ? cnt[w * a.L + tid] : 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) own.x += c[w];
        own.y = (own.x + kLmTile - 1) / kLmTile;
        scan = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int p = __shfl_up_sync(0xffffffffu, scan.x, off), q = __shfl_up_sync(0xffffffffu, scan.y, off);
            if (lane >= off) scan.x += p, scan.y += q;
        }
    }
    if (lane == 31) s_warp[warp] = some ? scan : make_int2(0, 0);
    __syncthreads();
    if (some) {
        int2 before = make_int2(0, 0);
        for (int w = 0; w < warp; ++w) before.x += s_warp[w].x, before.y += s_warp[w].y;
        if (tid < a.L) {
            int at = before.x + scan.x - own.x;
            first_row[tid] = at;
            first_tile[tid] = before.y + scan.y - own.y;
            if (tid == a.L - 1) {
                first_row[a.L] = at + own.x;
                first_tile[a.L] = before.y + scan.y;
            }
#pragma unroll
            for (int w = 0; w < 32; ++w) {
                cnt[w * a.L + tid] = static_cast<uint16_t>(at);
                at += c[w];
            }
        }
    }
    __syncthreads();
#pragma unroll 8
    for (int i = lo + lane; i < hi; i += 32) {
        const int e = sid[i];
        if (e != 0xffff) a.row_token[mine[e] + place[i]] = i;
    }
    const int all = first_tile[a.L];
    if (tid == 0) *a.ntiles = all;
    for (int i = tid; i < all; i += 1024) {
        int e = 0, behind = a.L;                // the adapter whose tiles hold i
        while (behind - e > 1) {
            const int mid = (e + behind) >> 1;
            if (first_tile[mid] <= i)
                e = mid;
            else
                behind = mid;
        }
        const int row0 = first_row[e] + (i - first_tile[e]) * kLmTile;
        a.tiles[i] = LmTile{e, row0, min(kLmTile, first_row[e + 1] - row0), 0};
        a.arrived[i] = 0;
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fetch) {   // else 16 zero bytes
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fetch ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A loading thread's share of a tile of 128 rows x 128 bytes: 16-byte piece
// `tid % 8` of rows tid / 8 + 16 i, the 128-byte swizzle applied by hand.  (A
// TMA gather of four such rows an instruction reached 1.6 TB/s here.)
struct RowLoader {
    int32_t token[8];
    int count, r0, piece;
    uint32_t at;
    __device__ __forceinline__ RowLoader(int tid)
        : count(0), r0(tid >> 3), piece(tid & 7),
          at(static_cast<uint32_t>((tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) << 4))) {}
    __device__ __forceinline__ void tile(const LmArgs& a, const LmTile& t) {
        count = t.count;
#pragma unroll
        for (int i = 0; i < 8; ++i) token[i] = r0 + 16 * i < count ? a.row_token[t.row0 + r0 + 16 * i] : 0;
    }
    // rows of `pitch` bytes, their bytes [byte0, byte0 + 128); past the pitch: zeros
    __device__ __forceinline__ void load(uint32_t dst, const void* base, size_t pitch, size_t byte0) const {
        const size_t b = byte0 + piece * 16;
        const bool in = b < pitch;
        const uint8_t* p = static_cast<const uint8_t*>(base) + (in ? b : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r0 + 16 * i < count) cp_async16(dst + at + 2048 * i, p + token[i] * pitch, in);
    }
};

__device__ __forceinline__ uint32_t lm_idesc(int n) {   // FP32 += BF16 x BF16, both K-major, M = 128
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kLmTile >> 4) << 24);
}

// A ring position: slot and phase parity.
struct Ring {
    int slot = 0, phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) slot = 0, phase ^= 1;
    }
};

// A warp's wait: one lane polls (a CTA of polling warps takes the issue slots of
// the one thread that feeds the tensor core: 50 against 47 us at 8192 x 8192).
__device__ __forceinline__ bool lm_wait_warp(uint64_t* bar, int parity) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait_bounded(bar, static_cast<uint32_t>(parity), kLmTimeout) ? 1 : 0;
    __syncwarp();
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Waits (bounded) until the last copy issued into each slot of a ring has landed.
__device__ __forceinline__ void lm_drain(uint64_t* full, int n, int issued) {
    for (int j = issued > n ? issued - n : 0; j < issued; ++j)
        mbar_wait_bounded(&full[j % n], static_cast<uint32_t>((j / n) & 1), kLmTimeout);
}

// The next part of v, which is left without it: the BF16 value next to v on the
// side of zero, v itself excluded.  So no part of a v other than 0 is 0 or has
// the other sign (down to where BF16 ends, 2^-133), and where B is infinite the
// parts' products add up to v's own infinity, not to NaN; nor does a v above the
// largest BF16 become infinite.  What is left is exact and at most one step of
// the part, 2^-7 of v: after two parts a third takes it whole.  An infinite v
// leaves infinity to the last part, NaN stays NaN.
__device__ __forceinline__ float lm_part(float& v) {
    const uint32_t bits = __float_as_uint(v);
    const float p = v == 0.0f ? 0.0f : __uint_as_float((bits - 1u) & 0xffff0000u);
    v -= p;
    return p;
}

// v of 16 ranks from group gi of one row: scaled, split, written as operand rows.
__device__ __forceinline__ void lm_write_v(const LmArgs& a, int tile, int gi, int row, float scale, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 16 * gi + i < a.R ? v[i] * scale : 0.0f;
    for (int p = 0; p < a.parts; ++p) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = p == a.parts - 1 ? pack_bf16x2_rn(make_float2(v[2 * i], v[2 * i + 1]))
                                    : pack_bf16x2_rn(make_float2(lm_part(v[2 * i]), lm_part(v[2 * i + 1])));
        uint16_t* dst = a.v + (((static_cast<size_t>(tile) * a.parts + p) * a.ks + gi / 4) * kLmTile + row) * kLmSlab +
                        gi % 4 * 16;
        st_v4(dst, make_uint4(w[0], w[1], w[2], w[3]));
        st_v4(dst + 8, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

// The tensor core cuts off what its FP32 accumulator cannot hold, always
// towards zero, so a long chain of MMAs drifts (512 of them, H = 8192: 1.7e-6 of
// the result in the mean; 64 of them: 6e-7).  After kLmChain steps (32 MMAs) the
// accumulator is added to registers with ordinary rounding: 2e-7.  GH: groups of
// 16 ranks of an epilogue thread (the eight warps halve the ranks).
template <int GH>
__global__ void __launch_bounds__(kLmThreads, 1) lora_shrink_kernel(const __grid_constant__ CUtensorMap amap,
                                                                 const LmArgs a) {
    extern __shared__ uint8_t lm_raw[];
    const uint32_t raw = smem_addr(lm_raw);
    uint8_t* ring = lm_raw + (((raw + 1023u) & ~1023u) - raw);
    __shared__ __align__(8) uint64_t full[kLmMaxStages], empty[kLmMaxStages], acc_full[2], acc_empty[2], done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_issued, s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = a.stages, a_bytes = a.rn * 128, stage_bytes = kLmStep * (kLmSlabBytes + a_bytes);
    const uint32_t cols = a.rn <= 16 ? 32u : a.rn <= 32 ? 64u : a.rn <= 64 ? 128u : 256u;   // two accumulators
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 128 + 1);        // the loading threads' rows and the TMA's A
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kLmEpiWarps);
        }
        mbar_init(&done, 1);
        s_issued = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    griddep_wait();
    griddep_launch();

    const int J = (a.H + kLmStep * kLmSlab - 1) / (kLmStep * kLmSlab);   // steps of a tile
    const int64_t U = static_cast<int64_t>(*a.ntiles) * J;
    const int64_t G = min(static_cast<int64_t>(gridDim.x), max(U / kLmLeast, min(U, static_cast<int64_t>(1))));
    const bool works = blockIdx.x < G;       // every working CTA has at least one step
    const int64_t u0 = works ? U * blockIdx.x / G : 0, u1 = works ? U * (blockIdx.x + 1) / G : 0;

    if (warp == 0) {
        if (lane == 0) {
            Ring r;
            int issued = 0, j = static_cast<int>(u0 % J), tile = static_cast<int>(u0 / J);
            int arow = u0 < u1 ? a.tiles[tile].adapter * a.R : 0;
            for (int64_t u = u0; u < u1; ++u, ++j) {
                if (j == J) {
                    j = 0;
                    arow = a.tiles[++tile].adapter * a.R;
                }
                if (issued >= S && !mbar_wait_bounded(&empty[r.slot], static_cast<uint32_t>(r.phase ^ 1), kLmTimeout)) break;
                mbar_arrive_expect_tx(&full[r.slot], static_cast<uint32_t>(kLmStep * a_bytes));
#pragma unroll
                for (int h = 0; h < kLmStep; ++h)
                    tma_load_2d(smem_addr(ring) + r.slot * stage_bytes + kLmStep * kLmSlabBytes + h * a_bytes, &amap,
                                (j * kLmStep + h) * kLmSlab, arow, &full[r.slot]);
                ++issued;
                r.next(S);
            }
            s_issued = issued;
        }
        __syncwarp();
    } else if (warp >= kLmLoadWarp) {
        RowLoader rows(threadIdx.x - kLmLoadWarp * 32);
        Ring r;
        int issued = 0;
        bool ok = true;
        const size_t pitch = static_cast<size_t>(a.H) * 2;
        for (int64_t u = u0; ok && u < u1;) {
            const int j0 = static_cast<int>(u % J), j1 = static_cast<int>(min(static_cast<int64_t>(J), j0 + (u1 - u)));
            rows.tile(a, a.tiles[u / J]);
            for (int j = j0; j < j1; ++j) {
                ok = issued < S || lm_wait_warp(&empty[r.slot], r.phase ^ 1);
                if (!ok) break;
#pragma unroll
                for (int h = 0; h < kLmStep; ++h)
                    rows.load(smem_addr(ring) + r.slot * stage_bytes + h * kLmSlabBytes, a.x, pitch,
                              static_cast<size_t>(j * kLmStep + h) * 128);
                cp_async_arrive(&full[r.slot]);
                ++issued;
                r.next(S);
            }
            u += j1 - j0;
        }
        cp_async_wait_all();
    } else if (warp == 1) {
        if (lane == 0) {
            Ring r;
            const uint32_t idesc = lm_idesc(a.rn);
            const uint64_t x_desc = smem_desc_sw128(smem_addr(ring)),
                           a_desc = smem_desc_sw128(smem_addr(ring) + kLmStep * kLmSlabBytes);
            bool ok = true;
            int seg = 0;
            for (int64_t u = u0; ok && u < u1; ++seg) {
                const int j0 = static_cast<int>(u % J);
                const int j1 = static_cast<int>(min(static_cast<int64_t>(min(J, j0 + kLmChain)), j0 + (u1 - u)));
                const int b = seg & 1;
                if (seg >= 2 && !mbar_wait_bounded(&acc_empty[b], static_cast<uint32_t>(((seg >> 1) - 1) & 1), kLmTimeout))
                    break;
                tc_fence_after();
                const uint32_t acc = tmem + b * (cols / 2);
                for (int j = j0; j < j1; ++j) {
                    ok = mbar_wait_bounded(&full[r.slot], static_cast<uint32_t>(r.phase), kLmTimeout);
                    if (!ok) break;
                    // the rows were written through the generic proxy, by copies that the barrier has seen land;
                    // the MMA reads through the async proxy
                    fence_proxy_async_smem();
                    tc_fence_after();
                    // descriptors count in 16 bytes; what a step adds stays inside their address field
                    const uint64_t dx = x_desc + static_cast<uint32_t>(r.slot * stage_bytes >> 4),
                                   da = a_desc + static_cast<uint32_t>(r.slot * stage_bytes >> 4);
#pragma unroll
                    for (int h = 0; h < kLmStep; ++h)
#pragma unroll
                        for (int k = 0; k < kLmSlab / 16; ++k)
                            mma_bf16(acc, dx + (h * kLmSlabBytes + 32 * k >> 4), da + (h * a_bytes + 32 * k >> 4), idesc,
                                     (j != j0 || h != 0 || k != 0) ? 1u : 0u);
                    mma_commit(&empty[r.slot]);
                    r.next(S);
                }
                if (!ok) break;
                mma_commit(&acc_full[b]);
                u += j1 - j0;
            }
            if (works)
                mma_commit(&done);
            else
                mbar_arrive(&done);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2, row = 32 * quad + lane;
        int seg = 0;
        for (int64_t u = u0; u < u1;) {
            const int tile = static_cast<int>(u / J), j0 = static_cast<int>(u % J);
            const int j1 = static_cast<int>(min(static_cast<int64_t>(J), j0 + (u1 - u)));
            const int adapter = a.tiles[tile].adapter;
            const float scale = a.scales != nullptr ? a.scales[adapter] : 1.0f;
            // the CTAs that share the tile: the last c with U c / G <= u, for its first and last slab
            const int64_t first = static_cast<int64_t>(tile) * J;
            const int c0 = static_cast<int>(((first + 1) * G - 1) / U), c1 = static_cast<int>(((first + J) * G - 1) / U);
            float v[GH][16];
#pragma unroll
            for (int g = 0; g < GH; ++g)
#pragma unroll
                for (int i = 0; i < 16; ++i) v[g][i] = 0.0f;
            bool ok = true;
            for (int j = j0; j < j1; j += kLmChain, ++seg) {
                const int b = seg & 1;
                ok = lm_wait_warp(&acc_full[b], (seg >> 1) & 1) && ok;
                tc_fence_after();
                const uint32_t acc = tmem + b * (cols / 2) + (static_cast<uint32_t>(32 * quad) << 16);
#pragma unroll
                for (int g = 0; g < GH; ++g) {
                    if (16 * (2 * g + half) >= a.rn) break;
                    float w[16];
                    tmem_ld16(acc + 16 * (2 * g + half), w);
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[g][i] += w[i];
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
            }
            // a wait that ran out ends all eight warps together: they share barriers
            if (!named_bar_and(1, kLmEpiWarps * 32, ok)) break;
            float* mine = a.part + (static_cast<size_t>(blockIdx.x) + tile) * a.R * kLmTile + row;
#pragma unroll
            for (int g = 0; g < GH; ++g) {
                const int gi = 2 * g + half;
                if (16 * gi >= a.rn) break;
                if (c0 == c1) {
                    lm_write_v(a, tile, gi, row, scale, v[g]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * gi + i < a.R) mine[(16 * gi + i) * kLmTile] = v[g][i];
                }
            }
            if (c0 != c1) {
                __threadfence();
                named_bar_sync(1, kLmEpiWarps * 32);
                if (warp == 4 && lane == 0) {
                    s_last = atomicAdd(&a.arrived[tile], 1) == c1 - c0;
                    __threadfence();
                }
                named_bar_sync(1, kLmEpiWarps * 32);
                if (s_last) {
                    for (int gi = half; gi < a.rn / 16; gi += 2) {
                        float t[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) t[i] = 0.0f;
                        for (int c = c0; c <= c1; c += 4) {     // the loads of four partials at a time
                            float w[4][16];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const float* p = a.part + (static_cast<size_t>(c + q) + tile) * a.R * kLmTile + row;
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    w[q][i] = c + q <= c1 && 16 * gi + i < a.R ? __ldcg(p + (16 * gi + i) * kLmTile) : 0.0f;
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q)
#pragma unroll
                                for (int i = 0; i < 16; ++i) t[i] += w[q][i];
                        }
                        lm_write_v(a, tile, gi, row, scale, t);
                    }
                }
            }
            u += j1 - j0;       // s_last is set again only behind the next tile's first barrier
        }
    }
    if (threadIdx.x == 0) mbar_wait_bounded(&done, 0u, kLmTimeout);
    __syncthreads();
    if (threadIdx.x == 0) lm_drain(full, S, s_issued);
    tc_fence_after();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, cols);
}

template <typename O>
__global__ void __launch_bounds__(kLmThreads, 1) lora_expand_kernel(const __grid_constant__ CUtensorMap vmap,
                                                                 const __grid_constant__ CUtensorMap bmap,
                                                                 const LmArgs a) {
    constexpr int kSubCols = 128 / sizeof(O);          // columns of a 128-byte row piece
    constexpr int kSubs = kLmCols / kSubCols;
    extern __shared__ uint8_t lm_raw[];
    const uint32_t raw = smem_addr(lm_raw);
    uint8_t* sv = lm_raw + (((raw + 1023u) & ~1023u) - raw);
    const int v_slabs = a.parts * a.ks;
    uint8_t* sb = sv + static_cast<size_t>(a.v_bufs) * v_slabs * kLmSlabBytes;
    uint8_t* sbase = sb + static_cast<size_t>(a.b_stages) * kLmSlabBytes;
    __shared__ __align__(8) uint64_t v_full[2], v_empty[2], b_full[kLmMaxStages], b_empty[kLmMaxStages],
        base_full[kLmMaxStages], base_empty[kLmMaxStages], acc_full[2], acc_empty[2], done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_issued[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t kCols = 2 * kLmCols;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kLmEpiWarps);
        }
        for (int i = 0; i < a.b_stages; ++i) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < a.base_stages; ++i) {
            mbar_init(&base_full[i], 128);
            mbar_init(&base_empty[i], kLmEpiWarps / 2);
        }
        mbar_init(&done, 1);
        s_issued[0] = s_issued[1] = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s_tmem, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // The plan was complete before the shrink kernel started, base and B before
    // that: they are fetched at once, only v waits for the shrink kernel.
    griddep_launch();

    const int C = (a.N + kLmCols - 1) / kLmCols;
    const int64_t U = static_cast<int64_t>(*a.ntiles) * C, G = gridDim.x;   // a CTA may get no item
    const int64_t u0 = U * blockIdx.x / G, u1 = U * (blockIdx.x + 1) / G;

    if (warp == 0) {
        if (lane == 0) {
            Ring rv, rb;
            int nv = 0, nb = 0, cur = -1, adapter = 0;
            bool ok = true;
            for (int64_t u = u0; ok && u < u1; ++u) {
                const int tile = static_cast<int>(u / C), n0 = static_cast<int>(u % C) * kLmCols;
                const bool first = tile != cur;
                if (first) {
                    cur = tile;
                    adapter = a.tiles[tile].adapter;
                }
                for (int s = 0; s < a.ks; ++s) {
                    ok = nb < a.b_stages || mbar_wait_bounded(&b_empty[rb.slot], static_cast<uint32_t>(rb.phase ^ 1), kLmTimeout);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&b_full[rb.slot], kLmSlabBytes);
                    tma_load_2d(smem_addr(sb + static_cast<size_t>(rb.slot) * kLmSlabBytes), &bmap, s * kLmSlab,
                                adapter * a.N + n0, &b_full[rb.slot]);
                    ++nb;
                    rb.next(a.b_stages);
                }
                if (!ok) break;
                if (first) {
                    if (nv == 0) griddep_wait();
                    ok = nv < a.v_bufs || mbar_wait_bounded(&v_empty[rv.slot], static_cast<uint32_t>(rv.phase ^ 1), kLmTimeout);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&v_full[rv.slot], static_cast<uint32_t>(v_slabs * kLmSlabBytes));
                    for (int i = 0; i < v_slabs; ++i)
                        tma_load_2d(smem_addr(sv + static_cast<size_t>(rv.slot * v_slabs + i) * kLmSlabBytes), &vmap, 0,
                                    (tile * v_slabs + i) * kLmTile, &v_full[rv.slot]);
                    ++nv;
                    rv.next(a.v_bufs);
                }
            }
            s_issued[0] = nv, s_issued[1] = nb;
        }
        __syncwarp();
    } else if (warp >= kLmLoadWarp) {
        RowLoader rows(threadIdx.x - kLmLoadWarp * 32);
        Ring rx;
        int nx = 0, cur = -1;
        bool ok = true;
        const size_t pitch = static_cast<size_t>(a.N) * sizeof(O);
        for (int64_t u = u0; ok && u < u1; ++u) {
            const int tile = static_cast<int>(u / C), n0 = static_cast<int>(u % C) * kLmCols;
            if (tile != cur) {
                cur = tile;
                rows.tile(a, a.tiles[tile]);
            }
            for (int s = 0; s < kSubs && n0 + s * kSubCols < a.N; ++s) {
                ok = nx < a.base_stages || lm_wait_warp(&base_empty[rx.slot], rx.phase ^ 1);
                if (!ok) break;
                rows.load(smem_addr(sbase) + rx.slot * kLmSlabBytes, a.base, pitch,
                          static_cast<size_t>(n0 + s * kSubCols) * sizeof(O));
                cp_async_arrive(&base_full[rx.slot]);
                ++nx;
                rx.next(a.base_stages);
            }
        }
        cp_async_wait_all();
    } else if (warp == 1) {
        if (lane == 0) {
            Ring rv, rb;
            const uint32_t idesc = lm_idesc(kLmCols);
            bool ok = true;
            int cur = -1, i = 0;
            uint32_t v = 0;
            for (int64_t u = u0; u < u1; ++u, ++i) {
                const int tile = static_cast<int>(u / C);
                const int b = i & 1;
                if (i >= 2 && !mbar_wait_bounded(&acc_empty[b], static_cast<uint32_t>(((i >> 1) - 1) & 1), kLmTimeout)) break;
                if (tile != cur) {
                    cur = tile;
                    if (!mbar_wait_bounded(&v_full[rv.slot], static_cast<uint32_t>(rv.phase), kLmTimeout)) break;
                    v = smem_addr(sv) + rv.slot * v_slabs * kLmSlabBytes;
                }
                tc_fence_after();
                uint32_t more = 0u;
                for (int s = 0; s < a.ks; ++s) {
                    ok = mbar_wait_bounded(&b_full[rb.slot], static_cast<uint32_t>(rb.phase), kLmTimeout);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sbs = smem_addr(sb) + rb.slot * kLmSlabBytes;
                    const int steps = (min(a.R - s * kLmSlab, kLmSlab) + 15) / 16;
                    // the small parts first: every step cuts off what the sum so far cannot hold, always towards
                    // zero, and the parts of a v have its sign
                    for (int p = a.parts - 1; p >= 0; --p)
                        for (int k = 0; k < steps; ++k) {
                            mma_bf16(tmem + b * kLmCols, smem_desc_sw128(v + (p * a.ks + s) * kLmSlabBytes + 32u * k),
                                     smem_desc_sw128(sbs + 32u * k), idesc, more);
                            more = 1u;
                        }
                    mma_commit(&b_empty[rb.slot]);
                    rb.next(a.b_stages);
                }
                if (!ok) break;
                mma_commit(&acc_full[b]);
                if (u + 1 == u1 || static_cast<int>((u + 1) / C) != tile) {
                    mma_commit(&v_empty[rv.slot]);
                    rv.next(a.v_bufs);
                }
            }
            if (u0 < u1)
                mma_commit(&done);
            else
                mbar_arrive(&done);
        }
        __syncwarp();
    } else if (warp < 4) {
        // rows of tokens without an adapter
        if (a.out != a.base) {
            // one row at a time to a warp: such tokens come in long runs
            const size_t row_bytes = static_cast<size_t>(a.N) * sizeof(O);
            const int64_t step = gridDim.x * 2;
            for (int64_t t0 = blockIdx.x * 2 + warp - 2; t0 < a.T; t0 += 32 * step) {
                const int64_t t = t0 + lane * step;
                const int id = t < a.T ? a.ids[t] : 0;
                uint32_t none = __ballot_sync(0xffffffffu, id < 0 || id >= a.L);
                for (; none != 0; none &= none - 1) {
                    const size_t at = static_cast<size_t>(t0 + (__ffs(none) - 1) * step) * row_bytes;
                    const uint8_t* src = static_cast<const uint8_t*>(a.base) + at;
                    uint8_t* dst = static_cast<uint8_t*>(a.out) + at;
#pragma unroll 8
                    for (size_t i = lane * 16; i < row_bytes; i += 512) st_v4(dst + i, ld_nc_v4(src + i));
                }
            }
        }
    } else {
        const int quad = warp & 3, grp = (warp - 4) >> 2, row = 32 * quad + lane;
        Ring rx;
        int cur = -1, i = 0, count = 0;
        int32_t token[8];          // of rows 32 quad + 4 it + lane / 8, which this lane writes a piece of
        for (int64_t u = u0; u < u1; ++u, ++i) {
            const int tile = static_cast<int>(u / C), n0 = static_cast<int>(u % C) * kLmCols;
            const int b = i & 1;
            if (tile != cur) {
                cur = tile;
                const LmTile t = a.tiles[tile];
                count = t.count;
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int r = 32 * quad + 4 * it + (lane >> 3);
                    token[it] = r < count ? a.row_token[t.row0 + r] : 0;
                }
            }
            bool ok = lm_wait_warp(&acc_full[b], (i >> 1) & 1);
            tc_fence_after();
            const uint32_t acc = tmem + b * kLmCols + (static_cast<uint32_t>(32 * quad) << 16);
            for (int s = 0; s < kSubs && n0 + s * kSubCols < a.N; ++s, rx.next(a.base_stages)) {
                if ((s & 1) != grp) continue;
                ok = lm_wait_warp(&base_full[rx.slot], rx.phase) && ok;
                if (!ok) break;
                const uint32_t tile_s = smem_addr(sbase) + rx.slot * kLmSlabBytes;
                const uint32_t mine = tile_s + row * 128;
#pragma unroll
                for (int h = 0; h < kSubCols / 32; ++h) {
                    float d[32];
                    tmem_ld32(acc + s * kSubCols + 32 * h, d);
                    if constexpr (sizeof(O) == 4) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t at = mine + ((c ^ (row & 7)) << 4);
                            const uint4 w = lds128(at);
                            const float2 lo = add2(make_float2(__uint_as_float(w.x), __uint_as_float(w.y)),
                                                   make_float2(d[4 * c], d[4 * c + 1]));
                            const float2 hi = add2(make_float2(__uint_as_float(w.z), __uint_as_float(w.w)),
                                                   make_float2(d[4 * c + 2], d[4 * c + 3]));
                            sts128(at, make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x),
                                                  __float_as_uint(hi.y)));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t at = mine + (((4 * h + c) ^ (row & 7)) << 4);
                            uint4 w = lds128(at);
                            w.x = pack_bf16x2_rn(add2(unpack_bf16x2(w.x), make_float2(d[8 * c], d[8 * c + 1])));
                            w.y = pack_bf16x2_rn(add2(unpack_bf16x2(w.y), make_float2(d[8 * c + 2], d[8 * c + 3])));
                            w.z = pack_bf16x2_rn(add2(unpack_bf16x2(w.z), make_float2(d[8 * c + 4], d[8 * c + 5])));
                            w.w = pack_bf16x2_rn(add2(unpack_bf16x2(w.w), make_float2(d[8 * c + 6], d[8 * c + 7])));
                            sts128(at, w);
                        }
                    }
                }
                __syncwarp();
                const int chunk = lane & 7, col = n0 + s * kSubCols + chunk * (16 / static_cast<int>(sizeof(O)));
#pragma unroll
                for (int it = 0; it < 8; ++it) {
                    const int r = 32 * quad + 4 * it + (lane >> 3);
                    const uint4 w = lds128(tile_s + r * 128 + ((chunk ^ (r & 7)) << 4));
                    if (r < count && col < a.N)
                        st_v4(static_cast<O*>(a.out) + static_cast<size_t>(token[it]) * a.N + col, w);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&base_empty[rx.slot]);
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
        }
    }
    if (threadIdx.x == 0) mbar_wait_bounded(&done, 0u, kLmTimeout);
    __syncthreads();
    if (threadIdx.x == 0) {
        lm_drain(v_full, a.v_bufs, s_issued[0]);
        lm_drain(b_full, a.b_stages, s_issued[1]);
    }
    griddep_wait();   // every CTA, also one without work: this kernel ends behind the shrink kernel
    tc_fence_after();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kCols);
}

int lm_most_tiles(int T, int L) { return (T + kLmTile - 1) / kLmTile + (L < T ? L : T); }
int lm_parts(bool bf16) { return bf16 ? 2 : 3; }
size_t lm_pad(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

bool lm_one_plan(int T, int L) { return T <= kLmPlanTokens && L <= kLmPlanAdapters; }

// The workspace of the many-token path, in order.
struct LmLayout {
    size_t offsets, row_idx, row_token, dispatch, tiles, ntiles, arrived, part, v, bytes;
};
LmLayout lm_layout(int T, int H, int R, int L) {
    LmLayout l;
    const size_t nt = static_cast<size_t>(lm_most_tiles(T, L)), ks = static_cast<size_t>((R + kLmSlab - 1) / kLmSlab);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t p = at;
        at += lm_pad(n);
        return p;
    };
    l.row_token = take(static_cast<size_t>(T) * 4);
    const bool big = !lm_one_plan(T, L);
    l.offsets = take(big ? (static_cast<size_t>(L) + 1) * 4 : 0);
    l.row_idx = take(big ? static_cast<size_t>(T) * 4 : 0);
    l.dispatch = take(big ? dispatch_workspace_bytes(T, L) : 0);
    l.tiles = take(nt * sizeof(LmTile));
    l.ntiles = take(4);
    l.arrived = take(nt * 4);
    l.part = take((nt + kLmCtas) * R * kLmTile * 4);
    l.v = take(nt * 3 * ks * kLmSlabBytes);
    l.bytes = at;
    return l;
}

cudaError_t lm_launch(const void* kernel, int grid, int threads, size_t smem, void** args, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_lora_many(const LoraLaunch& l, cudaStream_t s) {
    const LmLayout at = lm_layout(l.T, l.H, l.R, l.L);
    uint8_t* w = static_cast<uint8_t*>(l.workspace);
    LmArgs a{};
    int32_t* offsets = reinterpret_cast<int32_t*>(w + at.offsets);
    int32_t* row_idx = reinterpret_cast<int32_t*>(w + at.row_idx);
    int32_t* row_token = reinterpret_cast<int32_t*>(w + at.row_token);
    a.ids = l.ids, a.x = l.x, a.offsets = offsets, a.row_token = row_token;
    a.tiles = reinterpret_cast<LmTile*>(w + at.tiles);
    a.ntiles = reinterpret_cast<int32_t*>(w + at.ntiles);
    a.arrived = reinterpret_cast<int32_t*>(w + at.arrived);
    a.part = reinterpret_cast<float*>(w + at.part);
    a.v = reinterpret_cast<uint16_t*>(w + at.v);
    a.scales = l.scales, a.base = l.base, a.out = l.out;
    a.T = l.T, a.H = l.H, a.N = l.N, a.R = l.R, a.L = l.L;
    a.rn = (l.R + 15) / 16 * 16;
    a.ks = (l.R + kLmSlab - 1) / kLmSlab;
    a.parts = lm_parts(l.bf16);
    a.stages = kLmBytes / (kLmStep * (kLmSlabBytes + a.rn * 128));
    if (a.stages > kLmMaxStages) a.stages = kLmMaxStages;
    // the expand kernel's 13 slabs of 16 KB: v (twice while it is one slab wide), B, and the rest base
    a.v_bufs = a.ks == 1 ? 2 : 1;
    a.b_stages = a.ks == 1 ? 2 : 3;
    a.base_stages = kLmBytes / kLmSlabBytes - a.v_bufs * a.parts * a.ks - a.b_stages;
    CUtensorMap amap, vmap, bmap;
    constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    constexpr auto kSw = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t v_rows = static_cast<uint64_t>(lm_most_tiles(l.T, l.L)) * a.parts * a.ks * kLmTile;
    if (!encode_2d_map(&amap, kBf16, 2, l.a, static_cast<uint64_t>(l.L) * l.R, l.H, static_cast<uint64_t>(l.H) * 2,
                       static_cast<uint32_t>(a.rn), kLmSlab, kSw) ||
        !encode_2d_map(&vmap, kBf16, 2, a.v, v_rows, kLmSlab, kLmSlab * 2, kLmTile, kLmSlab, kSw) ||
        !encode_2d_map(&bmap, kBf16, 2, l.b, static_cast<uint64_t>(l.L) * l.N, l.R, static_cast<uint64_t>(l.R) * 2,
                       kLmCols, kLmSlab, kSw))
        return cudaErrorInvalidValue;
    cudaError_t e;
    void* targs[] = {&a};
    if (lm_one_plan(l.T, l.L)) {
        const void* plan = reinterpret_cast<const void*>(lora_plan_kernel);
        const size_t psmem = lm_plan_bytes(l.T, l.L);
        e = allow_smem(plan, psmem);
        if (e == cudaSuccess) e = lm_launch(plan, 1, 1024, psmem, targs, s);
    } else {
        e = launch_dispatch(l.ids, l.T, 1, 0, l.L, offsets, row_idx, row_token, w + at.dispatch, s);
        if (e == cudaSuccess) e = lm_launch(reinterpret_cast<const void*>(lora_tiles_kernel), 1, 1024, 0, targs, s);
    }
    if (e != cudaSuccess) return e;
    const int smem = kLmBytes + 1024;
    const void* const shrinks[] = {reinterpret_cast<const void*>(lora_shrink_kernel<1>),
                                   reinterpret_cast<const void*>(lora_shrink_kernel<2>),
                                   reinterpret_cast<const void*>(lora_shrink_kernel<3>),
                                   reinterpret_cast<const void*>(lora_shrink_kernel<4>)};
    const void* shrink = shrinks[(a.rn + 31) / 32 - 1];
    const void* expand = l.bf16 ? reinterpret_cast<const void*>(lora_expand_kernel<uint16_t>)
                                : reinterpret_cast<const void*>(lora_expand_kernel<float>);
    for (const void* k : {shrink, expand}) {
        e = allow_smem(k, static_cast<size_t>(smem));
        if (e != cudaSuccess) return e;
    }
    const int ctas = device_info().sm_count < kLmCtas ? device_info().sm_count : kLmCtas;
    void* sargs[] = {&amap, &a};
    e = lm_launch(shrink, ctas, kLmThreads, smem, sargs, s);
    if (e != cudaSuccess) return e;
    void* eargs[] = {&vmap, &bmap, &a};
    return lm_launch(expand, ctas, kLmThreads, smem, eargs, s);
}

}  // namespace

// Whether the one-launch path takes a batch: as far as its CTAs' threads look at
// the tokens, and with many ranks, whose columns its FP32 multiply-adds form,
// not quite so far (8192 -> 8192 on the GPU, few against many: rank 64, 128
// tokens 29 against 33 us, 256 tokens 47 against 31; rank 16, 256 tokens 16
// against 27).
static bool lora_few(int T, int R) { return T <= (R <= kLoraNarrow ? kLoraTokens : kLoraTokensWide); }

size_t lora_workspace_bytes(int T, int H, int N, int R, int L) {
    return lora_few(T, R) ? 0 : lm_layout(T, H, R, L).bytes;
}

cudaError_t launch_lora_add(const LoraLaunch& l, cudaStream_t s) {
    if (!lora_few(l.T, l.R)) return launch_lora_many(l, s);
    LoraArgs a{};
    a.T = l.T, a.H = l.H, a.N = l.N, a.R = l.R, a.L = l.L;
    a.x = l.x, a.a = l.a, a.b = l.b, a.ids = l.ids, a.scales = l.scales, a.base = l.base, a.out = l.out;
    a.kc = ((l.H + kLoraCluster - 1) / kLoraCluster + 31) / 32 * 32;
    a.nc = ((l.N + kLoraCluster - 1) / kLoraCluster + 7) / 8 * 8;
    if (l.R <= 16) return launch_lora_few<1>(a, l.bf16, s);
    if (l.R <= 32) return launch_lora_few<2>(a, l.bf16, s);
    if (l.R <= 64) return launch_lora_few<4>(a, l.bf16, s);
    return launch_lora_few<8>(a, l.bf16, s);
}

}  // namespace mb
