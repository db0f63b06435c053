// gdla_internal.h - launch plans shared between the C-ABI layer and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gdla {

// Prefill: one MMA tile = 24 tokens x 5 heads = 120 of the 128 MMA rows. The
// CTA size and key tile depend on the window (see prefill_geometry).
constexpr int kPrefillTileTokens = 24;
constexpr int kPrefillSlidingMaxWindow = 256;  // windows up to this use the sliding configuration

struct PrefillGeometry {
    int cta_tokens;       // tokens per CTA (a multiple of kPrefillTileTokens)
    int key_tile;         // keys per K/V tile
    int v_box;            // keys per V TMA box
    bool async_epilogue;  // gate/lambda/output tensor maps are used
};
PrefillGeometry prefill_geometry(int window);
constexpr int kPlanMaxSeqs = 256;    // sequences per launch (more are split across launches)
constexpr int kPlanMaxItems = 6144;  // q-tiles per launch
constexpr int kItemSeqShift = 20;
constexpr uint32_t kItemTileMask = (1u << kItemSeqShift) - 1u;

// Work item of a persistent CTA in its round r (0, 1, ...): the CTAs take the
// list round-robin, in reverse order on odd rounds, so that over a list sorted
// heaviest first every CTA gets a similar total (plain round-robin hands CTA 0
// the heaviest item of every round).
__device__ __forceinline__ int snake_item(int r) {
    const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return r * g + ((r & 1) ? g - 1 - c : c);
}

// The keys of a q tile whose window starts at kv_lo, with `sinks` first tokens visible behind it,
// as one run of columns that the key tiles cut: `pre` columns of sinks (the count rounded up to
// the 8 rows of a swizzle atom; the columns past it are masked), then the keys from kv_lo on.
// With the sinks in a tile of their own a q tile of the window-128 sliding schedule would visit four
// tiles instead of three; in the run, 48 tokens' 175 keys and up to 16 sinks are three
// (2 x 8192 tokens, 16 heads: 335 -> 299 us). Where the two would meet, one run from key 0 (pre = 0).
struct SinkRun {
    int pre, kv_lo;
};
__host__ __device__ __forceinline__ SinkRun sink_run(int kv_lo, int sinks) {
    const int pre = (sinks + 7) & ~7;
    if (kv_lo <= pre) return {0, sinks > 0 ? 0 : kv_lo};
    return {pre, kv_lo};
}
// Tensor maps of the tile in which sinks and window meet: pre % key_tile sink rows, then the rest.
template <bool SINK>
struct SinkMaps {};
template <>
struct SinkMaps<true> {
    CUtensorMap k_sink, k_rest, v_sink, v_rest;
};

// Tensor maps of V in boxes of 1, 2, 4, 8, 16 and 32 rows: the tile in which a sequence ends is loaded up to its last row
// with them, and filled with zeros (rows past the tensor) behind it. The whole tile's box would run on into the
// next sequence, whose weights here are zero; but zero times an infinity or a NaN is NaN.
struct EndMaps {
    CUtensorMap v[6];
};

// How the dK, dV kernel with sinks cuts its items (see the backward below).
struct DkvSplit {
    int chunks, chunk_steps, sink_steps;
};

// Passed by value (kernel parameters): the q-tiles of one launch, heaviest
// first. The host builds the largest form and launches the smallest capacity
// that holds the plan, so a launch carries 3.6, 9.2 or 28.7 KB (0.3, 0.5 or
// 2.1 KB of it the places of the partials, which only a backward with sinks reads).
template <int MAX_ITEMS, int MAX_SEQS>
struct PrefillPlanT {
    static constexpr int kMaxItems = MAX_ITEMS;
    static constexpr int kMaxSeqs = MAX_SEQS;
    int n_items;
    int hkv;
    int window;
    int sinks;                // first tokens visible behind the window (0 with window <= 0)
    int n_seqs;
    int n_rows;               // packed rows of the call
    int seq_start[MAX_SEQS];  // packed row of each sequence's first token
    int seq_len[MAX_SEQS];
    DkvSplit split;           // dkv with sinks
    int part[MAX_SEQS];       // .. the sequence's first sink partial, -1 for none
    int tile_part[MAX_SEQS];  // .. its first tile's first partial where tiles are cut
    uint32_t items[MAX_ITEMS];  // (local sequence << kItemSeqShift) | CTA block index
};
using PrefillPlan = PrefillPlanT<kPlanMaxItems, kPlanMaxSeqs>;
using PrefillPlanMedium = PrefillPlanT<2048, 64>;
using PrefillPlanSmall = PrefillPlanT<768, 32>;

// Backward: what the forward recompute leaves for the gradient kernels (and the
// gradients it finishes itself). Row statistics per (token, KV group): the
// base-2 log-sum-exp of the scaled scores of heads 0..4 (4 signal, noise) at
// 0..4, and rowsum(dH * H) of the same heads at 8..12.
constexpr int kBwdStats = 16;
struct BwdIO {
    const __nv_bfloat16 *dout;   // [N, 4H, 128]
    __nv_bfloat16 *dgate;        // [N, 4H, 128]
    float *dlambda;              // [N, 4H]
    __nv_bfloat16 *dh_sig;       // [N, 4H, 128]: gradient of H_S (= dout * sigmoid(gate)), bf16
    __nv_bfloat16 *dh_noise;     // [N, H, 128]: gradient of H_N, bf16
    float *stats;                // [N, H, kBwdStats]
};

struct PrefillLaunch {
    CUtensorMap tm_qs, tm_qn, tm_k, tm_v;
    SinkMaps<true> sink;                  // with sinks
    EndMaps end;
    CUtensorMap tm_gate, tm_lam, tm_out;  // used by the asynchronous epilogue (short windows)
    const float *lambda;
    const __nv_bfloat16 *gate;
    __nv_bfloat16 *out;
    BwdIO bwd;                            // backward recompute only
};

// Backward gradient kernels (gdla_prefill_bwd.cu). Plans: dq - items are 24-token
// q tiles (cost: 64-key tiles visited); dkv - items are 128-key tiles (cost:
// 12-token steps over the rows that see them).
constexpr int kBwdQKeyTile = 64;
constexpr int kBwdKeyTile = 128;
constexpr int kBwdStepTokens = 12;
struct BwdLaunch {
    CUtensorMap tm_qs, tm_qn;       // Q boxes of 6 tokens (as the forward)
    CUtensorMap tm_dhs, tm_dhn;     // dH boxes of 6 tokens
    CUtensorMap tm_qs12, tm_qn12;   // Q boxes of 12 tokens (dkv steps)
    CUtensorMap tm_dhs12, tm_dhn12; // dH boxes of 12 tokens
    SinkMaps<true> sink64;          // with sinks: of 64-key tiles (dq)
    CUtensorMap tm_k64, tm_v64;     // 64-key K / V boxes (dq)
    CUtensorMap tm_k128, tm_v128;   // 128-key K / V boxes (dkv)
    CUtensorMap tm_stats;           // row statistics, 12 tokens of one group
    const float *stats;
    __nv_bfloat16 *dq_sig, *dq_noise, *dk, *dv;
    float *part;                    // sinks: fp32 partials of dK | dV, [slot][KV head][sink][320]
    float *tile_part;               // .. of cut tiles, [slot][KV head][128][320]
};
// dK, dV with sinks. Every later token of a sequence sees them, so the rows past the first key
// tile's window are cut into chunks of sink_steps steps, an item each, whose sums for the
// sinks leave in fp32 and are added up in order by a last kernel. Where the key tiles are too few
// for the card, the tiles' own steps are cut the same way: `chunks` items per tile of chunk_steps
// steps, every row by way of partials. (5 sequences of 2,661 tokens, 2 heads, window 333: 46 items of
// up to 39 steps took 57 us.)
constexpr uint32_t kItemSinkChunk = 1u << 19;  // in a dkv item's tile index: sink chunk, not key tile
// Steps of the key tile at u0, and sink chunks behind those of the first tile.
__host__ __device__ __forceinline__ int bwd_tile_steps(int L, int u0, int window) {
    const int t_end = (window > 0 && window < L - u0 - (kBwdKeyTile - 1)) ? u0 + kBwdKeyTile - 1 + window : L;
    return (t_end - u0 + kBwdStepTokens - 1) / kBwdStepTokens;
}
__host__ __device__ __forceinline__ int bwd_sink_chunks(int L, int window, int sink_steps) {
    const int left = (L + kBwdStepTokens - 1) / kBwdStepTokens - bwd_tile_steps(L, 0, window);
    return left > 0 ? (left + sink_steps - 1) / sink_steps : 0;
}
constexpr int kSinkSumMaxSeqs = 256;
struct BwdSinkSum {  // the sequences of one launch of the last kernel
    const float *part, *tile_part;
    __nv_bfloat16 *dk, *dv;
    int hkv, sinks, n_seqs, window;
    DkvSplit split;
    int row0[kSinkSumMaxSeqs + 1];  // first row (key) of the launch that is the sequence's
    int start[kSinkSumMaxSeqs];     // packed row of its first token
    int len[kSinkSumMaxSeqs];
    int slot[kSinkSumMaxSeqs];      // its first sink partial (-1: none), and its first tile's first partial
    int tile_slot[kSinkSumMaxSeqs];
};
cudaError_t launch_bwd_sink_sum(const BwdSinkSum &sum, cudaStream_t stream);
cudaError_t launch_bwd_dq(const BwdLaunch &launch, const PrefillPlan &plan, cudaStream_t stream);
cudaError_t launch_bwd_dkv(const BwdLaunch &launch, const PrefillPlan &plan, cudaStream_t stream);

cudaError_t launch_prefill(const PrefillLaunch &launch, const PrefillPlan &plan, cudaStream_t stream);
// Backward, first pass: the forward recomputed on the forward's schedule for the
// plan's window (prefill_geometry), writing launch.bwd instead of the output.
cudaError_t launch_prefill_bwd_recompute(const PrefillLaunch &launch, const PrefillPlan &plan, cudaStream_t stream);

// SM count of a device, queried once per device and cached (0 on failure).
constexpr int kMaxCachedDevices = 64;
int device_sm_count(int dev);

// Identifier of the CUDA context current on the calling thread (0 if none is
// current or it cannot be read). Tearing the primary context down (a device
// reset) and re-creating it gives a new identifier, so host caches of facts
// that belong to a context (kernel attribute opt-ins, symbol addresses) key
// on it and are refreshed after a reset.
unsigned long long current_context_id();

// One flag per device, valid for one context: set() records the context it was
// set in, is_set() holds only while that context is still the current one.
struct PerContextFlag {
    std::atomic<unsigned long long> ctx[kMaxCachedDevices];
    bool is_set(int dev, unsigned long long id) const {
        return id != 0 && dev >= 0 && dev < kMaxCachedDevices && ctx[dev].load(std::memory_order_relaxed) == id;
    }
    void set(int dev, unsigned long long id) {
        if (id != 0 && dev >= 0 && dev < kMaxCachedDevices) ctx[dev].store(id, std::memory_order_relaxed);
    }
};

// Decode: split-KV.
constexpr int kDecodeMaxSplits = 64;
constexpr int kDecodeMinSplitKeys = 1024;

struct DecodePlan {
    int batch;
    int hkv;
    int window;
    int max_seqlen_k;
    int num_cache_rows;
    int num_splits;
    int split_keys;        // keys per split (multiple of 64)
    long long ml_offset_floats;  // start of the (m, l) area in the workspace, in floats
};

struct DecodeLaunch {
    CUtensorMap tm_k, tm_v;
    const __nv_bfloat16 *q_sig, *q_noise;
    const int32_t *cu_seqlens_k;
    const float *lambda;
    const __nv_bfloat16 *gate;
    __nv_bfloat16 *out;
    float *ws;
};

cudaError_t launch_decode(const DecodeLaunch &launch, const DecodePlan &plan, cudaStream_t stream);
int decode_smem_bytes();

// Decode over the latent cache: split-KV, then a combine with the W^UV up-projection.
constexpr int kLatentMaxSplits = 32;
constexpr int kLatentMinSplitKeys = 2048;

struct LatentPlan {
    int batch;
    int hkv;
    int window;
    int max_seqlen_k;
    int num_cache_rows;
    int num_splits;
    int split_keys;              // keys per split (multiple of the 48-key stage)
    long long ml_offset_floats;  // start of the (m, l) area in the workspace, in floats
};

struct LatentLaunch {
    CUtensorMap tm_qs, tm_qn, tm_c, tm_w;
    const int32_t *cu_seqlens_k;
    const float *lambda;
    const __nv_bfloat16 *gate;
    __nv_bfloat16 *out;
    float *ws;
};

LatentPlan make_latent_plan(int batch, int hkv, int max_seqlen_k, int window, int num_cache_rows);
size_t latent_workspace_bytes(const LatentPlan &plan);
cudaError_t launch_decode_latent(const LatentLaunch &launch, const LatentPlan &plan, cudaStream_t stream);

constexpr int kPlanSms = 148;  // SMs that the paged kernels' plans count on

// Paged KV cache: k_pages [num_pages, H, P, 192] and v_pages [num_pages, H, P, 128] in bf16,
// or in e4m3 with scales [num_pages, H]; block_table [batch, max_pages] names each
// sequence's pages in order. All pointers are device memory, strides in elements.
struct AppendPlan {
    const __nv_bfloat16 *k_nope, *k_rope, *v;
    long long nope_token, nope_head, rope_token, v_token, v_head;
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    const int32_t *block_table, *cu_new, *seqlens_k;
    int num_pages, page_size, page_shift, max_pages, num_tokens, batch, hkv;
    int heads_per_cta;  // set by the launch
    bool rotate;
};
cudaError_t launch_cache_append(const AppendPlan &plan, bool e4m3, cudaStream_t stream);

struct PagedDecode {
    const __nv_bfloat16 *q_sig, *q_noise;
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *seqlens_k;
    const float *lambda;
    const __nv_bfloat16 *gate;
    __nv_bfloat16 *out;
    float *ws;
    int num_pages, page_size, page_shift, max_pages, max_seqlen_k, batch, hkv, window, sinks;
    int splits, cluster;  // CTAs per (sequence, KV head), and how many of them form a cluster
    int warps;            // per CTA: 2, 4 or 8
    bool rotate;
};
struct PagedSplit {
    int cluster, parts;  // CTAs per cluster, clusters per (sequence, KV head)
    int warps;           // per CTA
};
PagedSplit paged_split(int batch, int hkv, int max_seqlen_k, int window, int sinks);
size_t paged_workspace_bytes(int batch, int hkv, const PagedSplit &split);
cudaError_t launch_decode_paged(const PagedDecode &plan, bool e4m3, cudaStream_t stream);

// Host-side decode split plan (shared by the workspace query and the launch).
DecodePlan make_decode_plan(int batch, int hkv, int max_seqlen_k, int window, int num_cache_rows);
size_t decode_workspace_bytes(const DecodePlan &plan);

}  // namespace gdla
