/*
 * fluxmi.h -- C ABI of libfluxmi: tile-granular GEMM fused with the
 * tensor-/expert-parallel data movement around it, for AMD Instinct MI355X
 * (gfx950), one GPU's share of the work.
 *
 * Operators (after the Flux README's five kernels, "快速开始"):
 *   fm_gemm              plain GEMM (the "gemm_only" reference point)
 *   fm_ag_gemm           AllGather fused with GEMM (dense MLP layer 0)
 *   fm_gemm_rs           GEMM fused with ReduceScatter (dense MLP layer 1)
 *   fm_moe_gather_gemm   token gather fused with grouped expert GEMM (MoE layer 0)
 *   fm_moe_gemm_scatter  grouped expert GEMM fused with top-k weighted
 *                        scatter-reduce (MoE layer 1)
 * and what stands around them in a sparse block: the router with its balance
 * loss (fm_moe_gate, fm_moe_gate_bwd), the norms, gate and residual add between
 * two blocks (fm_norm_residual, fm_norm_residual_bwd), and the products of a
 * decode step with 4-bit weights (fm_gemm_w4, fm_moe_gather_gemm_w4,
 * fm_moe_gemm_scatter_w4); in a dense block: dropout (fm_dropout), bias, dropout,
 * residual add and layer norm between two products (fm_layer_norm,
 * fm_layer_norm_bwd), and products in 8-bit integers (fm_quant_i8, fm_gemm_i8,
 * fm_linear_i8),
 * plus the AllGather variants fm_ag_gemm_pull (chunks read in place),
 * fm_ag_gemm_producers (copies done by workgroups of the same launch),
 * fm_moe_ag_gather_gemm (MoE layer 0 behind a token AllGather) with its
 * producer-workgroup and pull-mode forms (fm_moe_ag_gather_gemm_producers,
 * fm_moe_ag_gather_gemm_pull), the producer
 * half of the chunk-arrival protocol (fm_chunk_push, fm_chunk_push_dma,
 * fm_chunk_signal_paced) and the routing index on its own (fm_moe_route).
 *
 * Conventions for every call:
 *  - All matrices are dense and row-major.  A / X are [M, K]; B / W are [K, N].
 *  - Every pointer argument that names a matrix, flag, index buffer or
 *    workspace is a device pointer to memory owned by the caller; the library
 *    allocates nothing, keeps no state of its own between calls beyond cached
 *    device properties (the compute-unit count), and never synchronizes the
 *    host.  State that must outlive one call (the MoE operators' counters and
 *    completion flags) lives in a caller-owned workspace whose size
 *    fm_moe_workspace_bytes gives.  Calls are enqueued on `stream` (NULL =
 *    the null stream) and return before the work runs; every call is
 *    re-entrant for disjoint buffers.
 *  - 16-bit operands are IEEE binary16 (FM_F16) or bfloat16 (FM_BF16); every
 *    product is accumulated in fp32; narrowing to 16 bits rounds to nearest
 *    even.
 *  - Shape requirements: sizes >= 0; N and K multiples of 8; matrix pointers
 *    16-byte aligned.  A size of 0 in M or N makes the call a no-op; K == 0
 *    yields a zero product.
 *  - Errors: arguments are validated before anything is launched; an invalid
 *    call returns FM_ERR_INVALID_ARG or FM_ERR_UNSUPPORTED and enqueues no
 *    work.  FM_ERR_HIP means the launch itself failed.  A wait that gives up
 *    inside a kernel cannot be returned; it is written to `err_word` instead
 *    (see fm_ag_gemm).  No C++ exception crosses this interface.
 *  - Calls that write the same output on one stream are ordered; calls on
 *    different streams that write the same buffer race.
 *
 * Chunk-arrival protocol (fm_ag_gemm and its variants, fm_moe_ag_gather_gemm):
 *  - A producer makes a chunk's bytes visible device-wide before it publishes
 *    the chunk's flag.  The portable form is a store of the flag with release
 *    semantics at device (agent) scope, as fm_chunk_signal_paced does.  The
 *    library's own copy producers (fm_chunk_push, the producer workgroups of
 *    fm_ag_gemm_producers / fm_moe_ag_gather_gemm_producers) use an equivalent
 *    form that is cheaper on a GPU whose L2 caches are per XCD and not
 *    coherent with each other: each wave writes the chunk with write-through
 *    (system-scope) stores, waits until those stores have completed, passes a
 *    workgroup barrier, and only then updates the counter and the flag with
 *    relaxed atomics.  A release at agent scope would instead write back the
 *    whole L2 of the producer's XCD, once per workgroup.  Any producer must
 *    follow one of these two forms.  Consumers poll with relaxed loads and
 *    acquire at agent scope after the flag is seen.
 *  - The consumers of one launch may occupy every compute unit while they
 *    wait.  A producer kernel that runs on another stream (emulated arrival
 *    on one GPU) must therefore be enqueued on a stream that HIP maps to a
 *    different hardware queue than the consumer's, and before the consumer,
 *    so that its workgroups are dispatched first; with the default four
 *    hardware queues per process, streams created in a row take queues in
 *    turn.  A producer stream that shares the consumer's queue runs after
 *    the consumer, which then waits until spin_limit and reports
 *    FM_ERR_TIMEOUT.  Producers on the copy engines (fm_chunk_push_dma) and
 *    the producer workgroups of the *_producers forms (lowest workgroup ids,
 *    dispatched first) do not depend on this.
 */
#ifndef FLUXMI_H
#define FLUXMI_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fm_status {
    FM_OK = 0,
    FM_ERR_INVALID_ARG = 1,   /* null / misaligned pointer, bad size or count */
    FM_ERR_UNSUPPORTED = 2,   /* dtype combination or size the kernels do not cover */
    FM_ERR_HIP = 3,           /* the HIP launch failed */
    FM_ERR_TIMEOUT = 4        /* only ever written to err_word by a kernel */
} fm_status_t;

typedef enum fm_dtype {
    FM_F16 = 0,
    FM_BF16 = 1,
    FM_F32 = 2
} fm_dtype_t;

/* Activation applied to the fp32 result of MoE layer 0 (fm_moe_gather_gemm_act) or of
 * an 8-bit product (fm_gemm_i8) before it is rounded and stored. */
typedef enum fm_act {
    FM_ACT_NONE = 0,       /* H = X W1, as fm_moe_gather_gemm */
    FM_ACT_RELU = 1,       /* max(x, 0); of a NaN 0 in the MoE products, NaN in the 8-bit ones */
    FM_ACT_GELU_TANH = 2,  /* x/2 * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) */
    FM_ACT_SILU = 3        /* x / (1 + exp(-x)) */
} fm_act_t;

/* Library version, major*10000 + minor*100 + patch. */
int fm_version(void);

/* Static, human-readable name of a status code. */
const char* fm_status_str(fm_status_t status);

/*
 * fm_gemm -- C[M,N] = A[M,K] * B[K,N].
 * Defined by the GEMM in the FLUX review's MLP equations (section 三,
 * "MLP 前向传播"); it is also the non-split GEMM that the effective
 * communication time ECT = OverallTime - GEMM_non-split is measured against
 * (same review, "核心公式").
 *   ab   FM_F16 or FM_BF16: element type of A and B.
 *   c    FM_F16, FM_BF16 (same as ab) or FM_F32: element type of C.
 *   A    [M, K] row-major, B [K, N] row-major, C [M, N] row-major (written).
 * C must not overlap A or B.
 */
fm_status_t fm_gemm(fm_dtype_t ab, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                    const void* A, const void* B, void* C, hipStream_t stream);

/*
 * fm_ag_gemm -- Output1 = GEMM(AllGather(X), W1) with tile-granular overlap
 * (FLUX review, "MLP 前向传播" first GEMM and "AllGather 重叠": the gather and
 * the GEMM are split into tiles and fused in one kernel).
 *   X        [M, K] gathered activation buffer.  Row chunk c = rows
 *            [c*M/n_chunks, (c+1)*M/n_chunks) is written by a producer (a
 *            peer, or fm_chunk_push on another stream) and may be read only
 *            once flags[c] >= epoch.
 *   W        [K, N] weight shard; C [M, N] output (written), dt elements.
 *   n_chunks 1..64, and M % n_chunks == 0.
 *   flags    device array of n_chunks uint32 ready flags.  A producer writes
 *            the chunk, then publishes flags[c] = epoch with release
 *            semantics.  Epochs grow from call to call so flags never need
 *            resetting; the caller zero-fills them once.  In a HIP graph,
 *            whose replays repeat one epoch, zero the flags with a kernel
 *            (not a memset node) at the start of the graph instead.
 *   order    host array of n_chunks chunk indices, the expected arrival order
 *            (e.g. the local chunk first), or NULL for index order.  It only
 *            orders the tiles; the result does not depend on it.
 *   err_word device int32 or NULL.  If a wait exceeds spin_limit polls the
 *            kernel writes FM_ERR_TIMEOUT there, abandons its remaining tiles
 *            (C is then undefined) and exits; the call never hangs.
 *   spin_limit  polls before giving up (each poll sleeps ~0.1 us); 0 selects
 *            the default of 2^24 polls.
 * The result equals fm_gemm on the fully gathered X, bit for bit.
 */
fm_status_t fm_ag_gemm(fm_dtype_t dt, int64_t M, int64_t N, int64_t K, int32_t n_chunks,
                       const void* X, const void* W, void* C,
                       const uint32_t* flags, uint32_t epoch, const int32_t* order,
                       int32_t* err_word, int64_t spin_limit, hipStream_t stream);

/*
 * fm_ag_gemm_pull -- fm_ag_gemm in pull mode (FLUX review, "拉取 vs 推送数据
 * 传输": the compute tiles fetch the communicated data themselves).  No
 * gathered buffer exists: chunk c (rows [c*M/n_chunks, (c+1)*M/n_chunks) of
 * the gathered activation) is read in place from chunks[c], e.g. a peer's
 * buffer mapped into this process, once flags[c] >= epoch.
 *   chunks   host array of n_chunks device pointers, each to a 16-byte
 *            aligned [M/n_chunks, K] row-major block.
 *   W, C, n_chunks, flags, epoch, order, err_word, spin_limit  as fm_ag_gemm.
 * Row tiles are cut per chunk, so no tile reads two buffers; a chunk whose
 * row count is not a multiple of the tile height ends in a partial tile.
 * The result equals fm_gemm on the concatenated chunks, bit for bit.
 */
fm_status_t fm_ag_gemm_pull(fm_dtype_t dt, int64_t M, int64_t N, int64_t K, int32_t n_chunks,
                            const void* const* chunks, const void* W, void* C,
                            const uint32_t* flags, uint32_t epoch, const int32_t* order,
                            int32_t* err_word, int64_t spin_limit, hipStream_t stream);

/*
 * fm_ag_gemm_producers -- fm_ag_gemm with the data movement inside the same
 * launch, on workgroups of its own (COMET article, "COMET 的技术原理": thread
 * blocks are split into communication and computation roles, their ratio
 * adapted to the workload).  The first P workgroups of the grid are
 * producers: for each chunk in `order`, together they copy src[c] into rows
 * [c*M/n_chunks, (c+1)*M/n_chunks) of X and publish flags[c] = epoch
 * (release) once the whole chunk is in.  The other workgroups run the
 * AllGather-GEMM tiles, each after the flags of its chunks.  Producers take
 * the lowest workgroup ids and are dispatched first, so a waiting consumer
 * never holds back the producer it waits for.
 *   src          host array of n_chunks device pointers to [M/n_chunks, K]
 *                source blocks (a peer's chunk); NULL = chunk already in X
 *                (published at the start).  Sources must not overlap X.
 *   X            [M, K] gathered buffer (written by the producers, read by
 *                the consumers).
 *   counters     device uint32 [n_chunks], zero before the first call and
 *                left zero by every call.
 *   n_producers  P, a multiple of 8 (one per XCD per round) up to half the
 *                CUs; 0 picks the largest P that keeps the consumers' tile
 *                waves at their minimum, at most one per MiB copied (the
 *                per-shape choice of the producer:consumer ratio).
 *   W, C, flags, epoch, order, err_word, spin_limit  as fm_ag_gemm.
 * The result equals fm_gemm on the gathered X, bit for bit.
 */
fm_status_t fm_ag_gemm_producers(fm_dtype_t dt, int64_t M, int64_t N, int64_t K,
                                 int32_t n_chunks, const void* const* src, void* X,
                                 const void* W, void* C, uint32_t* flags, uint32_t* counters,
                                 uint32_t epoch, const int32_t* order, int32_t n_producers,
                                 int32_t* err_word, int64_t spin_limit, hipStream_t stream);

/*
 * fm_chunk_signal_paced -- emulated arrival at link speed: publish
 * flags[order[a]] = epoch (release, device scope) once arrive_ns[a]
 * nanoseconds have passed since this call's kernel started, for a = 0 ..
 * n_chunks-1.  The chunk data must already be in place (pull mode, or a
 * pre-filled gathered buffer); only the signals are timed, as a peer's
 * transfer over a link of known bandwidth would deliver them (the review's
 * "拉取 vs 推送数据传输" with the link as the only cost).  One workgroup of one
 * active lane, sleeping between signals, so it takes no measurable compute
 * from a kernel running beside it.
 *   order      host array, a permutation of 0..n_chunks-1, or NULL (index order).
 *   arrive_ns  host array of n_chunks non-decreasing times in [0, 1e9].
 * Times use the device's constant-rate wall clock (hipDeviceAttributeWallClockRate).
 */
fm_status_t fm_chunk_signal_paced(uint32_t* flags, int32_t n_chunks, const int32_t* order,
                                  const int64_t* arrive_ns, uint32_t epoch, hipStream_t stream);

/*
 * fm_chunk_push -- producer side of the chunk-arrival protocol: copy `bytes`
 * from src to dst, then publish *flag = epoch once every byte is visible
 * device-wide (the write-through form of the protocol above: every
 * workgroup's stores have completed before the last one to check in on
 * `counter` stores the flag).  This is what a peer rank's push (the review's
 * "推送模式" in "拉取 vs 推送数据传输") does to this rank's gathered buffer; on
 * one GPU src and dst are both local.
 *   bytes    multiple of 16 (0 = publish the flag only); src/dst 16-byte aligned
 *            and non-overlapping.
 *   counter  device uint32 scratch owned by the caller, zero before the
 *            first call and left zero after every call; one per flag in use.
 *   n_workgroups  copy workgroups, 0 = default (one per 96 KiB, at most
 *                 two per compute unit).
 */
fm_status_t fm_chunk_push(const void* src, void* dst, int64_t bytes, uint32_t* flag,
                          uint32_t* counter, uint32_t epoch, int32_t n_workgroups,
                          hipStream_t stream);

/*
 * fm_chunk_push_dma -- the same producer step on the copy engines: an
 * asynchronous device-to-device copy that uses no compute units, followed on
 * `stream` by a write of epoch into *flag made once the copy has completed.
 * This is how a peer's DMA engine delivers a chunk over a link and then rings
 * the signal (the review's push mode in "拉取 vs 推送数据传输"; the FlagCX
 * guide's put-with-signal), so the consumer's compute units are not spent on
 * the emulated transfer.
 *   bytes  multiple of 16 (0 = write the flag only); src/dst 16-byte aligned
 *          and non-overlapping; flag 4-byte aligned device memory.
 * Returns FM_ERR_HIP if the runtime rejects the copy or the flag write.
 */
fm_status_t fm_chunk_push_dma(const void* src, void* dst, int64_t bytes, uint32_t* flag,
                              uint32_t epoch, hipStream_t stream);

/*
 * fm_gemm_rs -- Output2 = ReduceScatter(GEMM(Output1, W2)), this rank's part
 * (FLUX review, "MLP 前向传播" second GEMM and "ReduceScatter 重叠").
 *   A        [M, K] (K = this rank's shard of the reduction), W [K, N].
 *   dst      host array of n_ranks device pointers; dst[r] is the fp32
 *            [M/n_ranks, N] slice owned by rank r and already holds the other
 *            ranks' partial sums.  The call adds (A*W)[rows of r] into dst[r]
 *            for every r: dst[r] += partial.
 *   n_ranks  1..16, M % n_ranks == 0; rank in [0, n_ranks).
 *            Tiles are taken slice by slice starting at (rank+1) % n_ranks
 *            (the review's tile-coordinate swizzling, "瓦片坐标 Swizzling").
 *   atomic   0: plain read-add-write (this call is the only writer of dst);
 *            1: fp32 atomic adds (several concurrent writers allowed).
 *   dt       FM_F16 or FM_BF16 for A and W.
 */
fm_status_t fm_gemm_rs(fm_dtype_t dt, int64_t M, int64_t N, int64_t K, int32_t n_ranks,
                       int32_t rank, const void* A, const void* W, float* const* dst,
                       int32_t atomic, hipStream_t stream);

/*
 * fm_moe_workspace_bytes -- bytes of device workspace that the MoE operators
 * (fm_moe_route, fm_moe_gather_gemm and its variants, fm_moe_gemm_scatter)
 * need for T tokens with topk pairs each, a hidden size `hidden` and n_local
 * local experts; 0 if the arguments are out of range (T < 0, topk < 1,
 * hidden < 0, n_local outside 1..64).  A workspace of this size serves every
 * call of one MoE layer with these (or smaller) sizes.
 * The workspace is 16-byte aligned device memory owned by the caller.  Fill
 * it with zeros once, before its first use; every call leaves it ready for
 * the next (calls keep an epoch and a few counters in it, so that nothing
 * needs resetting between calls, also when a call is replayed from a HIP
 * graph).  One workspace must not be used by two routes (or two combines) at
 * the same time: issue such calls on one stream, or order their streams.  A
 * route (or layer 0) and a combine may share one workspace concurrently.
 * Separate MoE layers (for instance two expert-parallel ranks emulated on one
 * GPU) that run at the same time need one workspace each.
 */
size_t fm_moe_workspace_bytes(int64_t T, int32_t topk, int64_t hidden, int32_t n_local);

/*
 * fm_moe_route -- expert-sorted row index of this rank's local experts
 * (COMET article, "COMET 的技术原理": the tensor shared between the MoE
 * layers is decomposed along the token dimension).
 *   topk_ids      device int32 [T, topk]: expert of pair p = t*topk + k.
 *   expert_begin  first local expert; local experts are
 *                 [expert_begin, expert_begin + n_local), n_local 1..64.
 *   expert_offsets  device int32 [n_local+1] (written): exclusive prefix sum
 *                 of the local per-expert pair counts.
 *   sorted_pairs  device int32 [T*topk] (written): positions
 *                 [0, expert_offsets[n_local]) hold the local pair ids stably
 *                 sorted by expert (increasing pair id within an expert); the
 *                 rest is left untouched.
 *   ws, ws_bytes  the MoE workspace (fm_moe_workspace_bytes); the per-chunk
 *                 histograms of the counting sort live there.  A null,
 *                 misaligned or too small workspace gives FM_ERR_INVALID_ARG.
 * Deterministic: identical bits on every call.
 */
fm_status_t fm_moe_route(int64_t T, int32_t topk, int32_t expert_begin, int32_t n_local,
                         const int32_t* topk_ids, int32_t* sorted_pairs,
                         int32_t* expert_offsets, void* ws, size_t ws_bytes,
                         hipStream_t stream);

/*
 * fm_moe_gather_gemm -- MoE layer 0 on this rank: route (as fm_moe_route),
 * then for local expert e and its j-th pair p:
 *   H[expert_offsets[e] + j, :] = X[p / topk, :] * W1[e]
 * (Flux README: grouped GEMM of MoE MLP layer 0; the token gather is fused
 * into the GEMM's A loads).  Row counts stay on the device: no host sync.
 *   X   [T, hidden]; W1 [n_local, hidden, ffn]; H [T*topk, ffn] (rows past
 *       expert_offsets[n_local] are left untouched).  dt FM_F16 or FM_BF16.
 *       With hidden = 0 the sum over K is empty: the local rows of H become
 *       0, and X and W1 may be null.  With T = 0 or ffn = 0 only the route
 *       runs.
 *   ws, ws_bytes  the MoE workspace, as fm_moe_route.
 */
fm_status_t fm_moe_gather_gemm(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                               int32_t topk, int32_t expert_begin, int32_t n_local,
                               const void* X, const int32_t* topk_ids, const void* W1,
                               void* H, int32_t* sorted_pairs, int32_t* expert_offsets,
                               void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * fm_moe_gather_gemm_act -- fm_moe_gather_gemm with an activation fused into
 * the epilogue: H[row, :] = act(X[p / topk, :] * W1[e]), the activation taken
 * in fp32 on the accumulated value, then rounded (RNE) to dt.  The FLUX
 * review's MLP forward pass (section 三, "MLP 前向传播") feeds the first GEMM's
 * output to the second as is, which is FM_ACT_NONE; the other forms cover
 * expert MLPs that apply an activation between their two GEMMs.  Arguments,
 * layouts and errors as fm_moe_gather_gemm; an act outside fm_act_t gives
 * FM_ERR_INVALID_ARG before anything is launched.
 */
fm_status_t fm_moe_gather_gemm_act(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                                   int32_t topk, int32_t expert_begin, int32_t n_local,
                                   const void* X, const int32_t* topk_ids, const void* W1,
                                   void* H, int32_t* sorted_pairs, int32_t* expert_offsets,
                                   fm_act_t act, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * fm_moe_ag_gather_gemm -- fm_moe_gather_gemm behind a token AllGather (Flux
 * README: all-gather fused with the grouped GEMM of MoE MLP layer 0): X is
 * the gathered token buffer of n_chunks expert-parallel ranks, chunk c
 * holding tokens [c*T/n_chunks, (c+1)*T/n_chunks), and a tile reads its token
 * rows only after every chunk they come from has flags[c] >= epoch (the
 * protocol of fm_ag_gemm; producers as fm_chunk_push / fm_chunk_push_dma).
 * Rows of an expert are sorted by token, so a tile needs the chunks between
 * its first and last token.  Tiles run in bands of a few M-tiles of one
 * expert, ordered by the expected arrival of the last chunk a band needs, so
 * the rows of the local and earliest chunks start before the others land.
 * topk_ids covers all T tokens and must be complete before the call.
 *   n_chunks  1..64, T % n_chunks == 0; flags device uint32 [n_chunks].
 *   order     host array of n_chunks chunk indices, the expected arrival
 *             order, or NULL for index order (as fm_ag_gemm; it only orders
 *             the tiles).
 *   err_word, spin_limit  as fm_ag_gemm (a wait past the limit writes
 *             FM_ERR_TIMEOUT there; H is then undefined).
 *   ws, ws_bytes  the MoE workspace, as fm_moe_route.
 * The result equals fm_moe_gather_gemm on the fully gathered X, bit for bit.
 */
fm_status_t fm_moe_ag_gather_gemm(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                                  int32_t topk, int32_t expert_begin, int32_t n_local,
                                  const void* X, const int32_t* topk_ids, const void* W1,
                                  void* H, int32_t* sorted_pairs, int32_t* expert_offsets,
                                  int32_t n_chunks, const uint32_t* flags, uint32_t epoch,
                                  const int32_t* order, int32_t* err_word, int64_t spin_limit,
                                  void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * fm_moe_ag_gather_gemm_producers -- fm_moe_ag_gather_gemm with the token
 * AllGather done inside the same launch by producer workgroups (COMET
 * article, "COMET 的技术原理": communication and computation thread blocks
 * of one fused MoE kernel).  The first P workgroups copy src[c] into token
 * rows [c*T/n_chunks, (c+1)*T/n_chunks) of X, chunks taken in `order`, and
 * publish flags[c] = epoch once a chunk is complete; the other workgroups
 * run the layer-0 tiles behind those flags, in the arrival-ordered bands of
 * fm_moe_ag_gather_gemm.  Producers hold the lowest workgroup ids and are
 * dispatched first.
 *   X            [T, hidden] gathered token buffer (written by the producers).
 *   src          host array of n_chunks device pointers to [T/n_chunks, hidden]
 *                blocks; NULL = chunk already in X (published at the start).
 *                Sources are 16-byte aligned and do not overlap X.
 *   counters     device uint32 [n_chunks], zero before the first call and
 *                left zero by every call.
 *   n_producers  P: a multiple of 8, 8 .. half the CUs; 0 = one per ~5 MiB
 *                copied, 8..64.
 *   the rest     as fm_moe_ag_gather_gemm.
 * The result equals fm_moe_gather_gemm on the gathered X, bit for bit.
 */
fm_status_t fm_moe_ag_gather_gemm_producers(
    fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn, int32_t topk, int32_t expert_begin,
    int32_t n_local, void* X, const int32_t* topk_ids, const void* W1, void* H,
    int32_t* sorted_pairs, int32_t* expert_offsets, int32_t n_chunks, const void* const* src,
    uint32_t* flags, uint32_t* counters, uint32_t epoch, const int32_t* order,
    int32_t n_producers, int32_t* err_word, int64_t spin_limit, void* ws, size_t ws_bytes,
    hipStream_t stream);

/*
 * fm_moe_ag_gather_gemm_pull -- fm_moe_ag_gather_gemm in pull mode (FLUX
 * review, "拉取 vs 推送数据传输"): no gathered token buffer; each layer-0 tile
 * reads its token rows in place from the owners' chunk buffers (on a node, the
 * peers' activations mapped into this process), after their flags.  Only the
 * tokens routed to this rank's experts are ever read.
 *   chunks  host array of n_chunks device pointers; chunks[c] is the
 *           16-byte aligned [T/n_chunks, hidden] block of tokens
 *           [c*T/n_chunks, (c+1)*T/n_chunks).
 *   the rest  as fm_moe_ag_gather_gemm (flags, epoch, order, err_word,
 *           spin_limit, ws; signals from fm_chunk_signal_paced or a peer).
 * The result equals fm_moe_gather_gemm on the concatenated chunks, bit for
 * bit.
 */
fm_status_t fm_moe_ag_gather_gemm_pull(
    fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn, int32_t topk, int32_t expert_begin,
    int32_t n_local, const void* const* chunks, const int32_t* topk_ids, const void* W1, void* H,
    int32_t* sorted_pairs, int32_t* expert_offsets, int32_t n_chunks, const uint32_t* flags,
    uint32_t epoch, const int32_t* order, int32_t* err_word, int64_t spin_limit, void* ws,
    size_t ws_bytes, hipStream_t stream);

/*
 * fm_moe_gemm_scatter -- MoE layer 1 on this rank with the top-k weighted
 * combine fused into the GEMM epilogue (Flux README: grouped GEMM fused with
 * the reduce-scatter of MoE MLP layer 1; COMET article, "COMET 的技术原理":
 * the per-token combine over the experts):
 *   out[t, :] += sum over local pairs p = t*topk + k of
 *                topk_weights[p] * (H[row(p), :] * W2[e(p)])
 * where row(p) is p's position in sorted_pairs (from fm_moe_gather_gemm /
 * fm_moe_route with the same arguments).
 *   H [rows, ffn] with rows = expert_offsets[n_local]; W2 [n_local, ffn, hidden];
 *   topk_weights device fp32 [T, topk]; out device fp32 [T, hidden].  With
 *   ffn = 0 the sum over K is empty (each local pair adds weight x 0) and H
 *   and W2 may be null; with T = 0 or hidden = 0 nothing is launched.
 *   Precondition: the local pairs of one token lie in different experts (a
 *   top-k choice never picks one expert twice).  A token with two pairs in
 *   one local expert is reported as FM_ERR_INVALID_ARG in err_word; the
 *   adds of the row tiles that hold the repeated pair are skipped, and out
 *   is then undefined.
 *   err_word  device int32 or NULL: receives FM_ERR_TIMEOUT if an ordering
 *             wait exceeds spin_limit polls (the launch then abandons its
 *             remaining tiles, out is undefined, the call never hangs), or
 *             FM_ERR_INVALID_ARG as above.  Left untouched otherwise.
 *   spin_limit  polls of one completion flag before giving up (each poll
 *             sleeps ~0.1 us); 0 selects the default of 2^24.
 *   ws, ws_bytes  the MoE workspace (fm_moe_workspace_bytes with the same T,
 *             topk, hidden and n_local or larger); FM_ERR_INVALID_ARG if it
 *             is null, misaligned or too small.
 * The additions into a token row are applied in local-expert order with plain
 * fp32 loads and stores (no atomics), so the result is deterministic.  Each
 * row tile of one expert waits for the tiles of earlier experts in its column
 * whose token ranges overlap its own, through per-(row tile, column tile)
 * completion flags in the workspace, stamped with an epoch that the kernel
 * itself advances there (so the call may be captured in a HIP graph and
 * replayed).  Tiles are handed out by atomic tickets from per-column queues
 * (one per pair of XCDs, each in expert order), so a tile only ever waits for
 * tiles that running workgroups hold: the call completes whatever share of
 * the GPU it gets (another kernel, or another combine on another stream with
 * its own workspace, may run beside it).
 */
fm_status_t fm_moe_gemm_scatter(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                                int32_t topk, int32_t n_local, const void* H, const void* W2,
                                const int32_t* sorted_pairs, const int32_t* expert_offsets,
                                const float* topk_weights, float* out, int32_t* err_word,
                                int64_t spin_limit, void* ws, size_t ws_bytes,
                                hipStream_t stream);

/*
 * fm_moe_gemm_scatter_noalloc -- fm_moe_gemm_scatter for callers that cannot
 * allocate or own a workspace (code under HIP graph capture, tight serving
 * loops, harnesses that forbid device allocation).  The combine's control
 * words and completion flags live in a static device array of the library,
 * 256 KiB per GPU, held until the process ends (its address is looked up, and
 * the array zero-filled by a kernel on `stream`, on the first call on each
 * GPU); the call itself allocates nothing.
 *   Arguments, results and errors as fm_moe_gemm_scatter without (ws,
 *   ws_bytes); the result is bit-identical to it.
 *   Limit: (ceil(T*topk/128) + n_local) * ceil(hidden/128) <= 65216, else
 *   FM_ERR_UNSUPPORTED (the EP=8 workload, T = 16384, top-2, hidden 4096,
 *   8 local experts, needs 8448).  FM_ERR_HIP if the array's address cannot
 *   be obtained.
 *   Every call on one GPU shares that GPU's array: calls that overlap in time
 *   on one GPU (two streams) race and give undefined results; issue them on
 *   one stream, or order the streams.
 */
fm_status_t fm_moe_gemm_scatter_noalloc(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                                        int32_t topk, int32_t n_local, const void* H,
                                        const void* W2, const int32_t* sorted_pairs,
                                        const int32_t* expert_offsets,
                                        const float* topk_weights, float* out,
                                        int32_t* err_word, int64_t spin_limit,
                                        hipStream_t stream);

/*
 * fm_moe_gate -- router of an MoE layer: the experts and weights of each token
 * from its router logits, and the layer's expert counts and balance loss.
 * With x = logits[t, :] in fp32 and
 *   u = x           (FM_GATE_SOFTMAX)      share = softmax(u) over all experts
 *   u = log s(x)    (FM_GATE_SIGMOID)      s(x) = 1 / (1 + exp(-x))
 * the score of an expert is share (softmax) or s(x) (sigmoid), and
 *   topk_ids[t, :]      the topk experts with the largest key, largest first,
 *                       equal keys by the lower expert.  The key is x, or with
 *                       a bias score + bias, evaluated in 64 bits.
 *   topk_weights[t, :]  scale * score of these experts or, renormalized,
 *                       scale * softmax of u over the chosen ones.
 *   counts[e]           slots of topk_ids that name expert e; counts[E] the
 *                       number of tokens that are not masked, n.
 *   prob_sums[e]        sum of share[t, e] over the tokens not masked.
 *   loss                E / (topk n^2) * sum_e counts[e] * prob_sums[e]; 1 for
 *                       perfectly even experts, 0 if n = 0.
 * topk_ids and topk_weights are what fm_moe_route and fm_moe_gemm_scatter take.
 *   dt, logits  FM_F16, FM_BF16 or FM_F32, [T, n_experts]; n_experts 1..1024.
 *               An expert with logit -inf is closed: it is never chosen, and
 *               its share is 0.  A slot that finds no open expert gets id -1
 *               and weight 0, which every MoE call here passes over.  A key
 *               that is NaN or -inf is never chosen.  A NaN among a row's
 *               logits (or +inf under a softmax) makes its shares NaN, and so
 *               prob_sums, the loss and its row of d_logits.  Without a bias,
 *               or with sigmoid scores, the row's other experts are chosen as
 *               ever; with a bias under a softmax every key of the row is made
 *               of those shares, and no slot finds an expert.
 *   topk        1..16 and <= n_experts.
 *   bias        fp32 [n_experts] or NULL; it only moves the choice.
 *   token_mask  uint8 [T] or NULL: tokens with 0 are padding.  Their logits are
 *               not used, their ids are -1 and their weights 0.
 *   counts      int32 [n_experts + 1], prob_sums fp32 [n_experts], loss fp32
 *               [1]: all three written, or all three NULL (then no workspace
 *               is needed).
 *   ws, ws_bytes  scratch of fm_moe_gate_workspace_bytes, 16-byte aligned; its
 *               contents need no preparation.  Calls that may run at the same
 *               time, captured graphs' replays among them, need one each.
 * Deterministic: identical bits on every call.
 */
typedef enum fm_gate_score { FM_GATE_SOFTMAX = 0, FM_GATE_SIGMOID = 1 } fm_gate_score_t;

size_t fm_moe_gate_workspace_bytes(int64_t T, int32_t n_experts);

fm_status_t fm_moe_gate(fm_dtype_t dt, int64_t T, int32_t n_experts, int32_t topk,
                        fm_gate_score_t score, int32_t renormalize, float scale,
                        const void* logits, const float* bias, const uint8_t* token_mask,
                        int32_t* topk_ids, float* topk_weights, int32_t* counts,
                        float* prob_sums, float* loss, void* ws, size_t ws_bytes,
                        hipStream_t stream);

/*
 * fm_moe_gate_bwd -- gradient of fm_moe_gate's weights and loss: d_logits from
 * d_weights (gradient of topk_weights) and d_loss (gradient of the loss).  The
 * choice of experts, the counts and the bias carry no gradient.
 *   topk_ids   as fm_moe_gate left them: slots outside [0, n_experts) take no
 *              part; a repeated expert adds up.
 *   d_weights  fp32 [T, topk], or NULL: no gradient by that way.
 *   counts     int32 [n_experts + 1] and d_loss, a device fp32, or both NULL.
 *              With counts (and n) summed over data-parallel ranks this is the
 *              gradient of the loss of the whole batch.
 *   d_logits   [T, n_experts] in dt (written whole: 0 for masked tokens and
 *              closed experts).  It must not overlap logits.
 *   the rest   as fm_moe_gate.
 */
fm_status_t fm_moe_gate_bwd(fm_dtype_t dt, int64_t T, int32_t n_experts, int32_t topk,
                            fm_gate_score_t score, int32_t renormalize, float scale,
                            const void* logits, const uint8_t* token_mask,
                            const int32_t* topk_ids, const float* d_weights,
                            const int32_t* counts, const float* d_loss, void* d_logits,
                            hipStream_t stream);

/*
 * fm_norm_residual -- what lies between two blocks of a residual stream: the
 * norm after a block, its gate and scale, the residual add and the norm before
 * the next block, in one pass.  For each row
 *   b   = block                               or, with w_post,
 *         block / rms(block) * w_post         rms(v) = sqrt(mean(v^2) + eps)
 *   out = resid + scale * gate * b
 *   y   = out / rms(out) * w_pre
 * all in fp32 (y from the fp32 value of out), rounded once when stored.  block
 * may be a slice that fm_gemm_rs filled or the combine's out (fp32); y is the
 * 16-bit input of fm_ag_gemm, fm_chunk_push or fm_moe_gather_gemm.
 *   dt         FM_F16 or FM_BF16: y, w_post, w_pre and gate.
 *   stream_dt  resid and out: dt or FM_F32.   block_dt  block: dt or FM_F32.
 *   M, N       rows and row length; N a multiple of 8, at most 16384.
 *   block      [M, N] or NULL: no block (out = resid; w_post and gate must be
 *              NULL too).   resid  [M, N] or NULL: 0.  Not both NULL.
 *   w_post, w_pre  [N] or NULL: no norm there.  y is NULL if and only if w_pre is.
 *   gate       [n_gates, N] or NULL: 1.  Row i takes gate row i / (M / n_gates);
 *              M is a multiple of n_gates (1: one for all, M: one per row,
 *              else one for each sequence of M / n_gates rows).
 *   out        [M, N] or NULL (not wanted); it may be resid itself.
 *   rstd_post, rstd_pre  fp32 [M] or NULL: 1 / rms, which the backward needs.
 */
fm_status_t fm_norm_residual(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                             int64_t N, const void* block, const void* resid, const void* w_post,
                             const void* w_pre, const void* gate, int64_t n_gates, float scale,
                             float eps, void* out, void* y, float* rstd_post, float* rstd_pre,
                             hipStream_t stream);

/*
 * fm_norm_residual_bwd -- gradients of fm_norm_residual.
 *   d_y      [M, N] dt, gradient of y; NULL if and only if w_pre is.
 *   d_out    [M, N] stream_dt, gradient of out from its later uses, or NULL: 0.
 *   out      [M, N] stream_dt as the forward stored it; needed with w_pre.
 *   block    [M, N] block_dt; needed for d_gate, d_w_post and, with w_post, for
 *            d_block.
 *   rstd_post  as the forward stored it; needed where w_post is given and block
 *            is needed.   rstd_pre  the same; needed with w_pre.
 *   d_resid  [M, N] stream_dt or NULL: gradient of resid (of out in total).
 *            It may be d_out itself.
 *   d_block  [M, N] block_dt or NULL.
 *   d_w_post, d_w_pre fp32 [N], d_gate fp32 [n_gates, N]: written whole, or
 *            NULL; each only beside its weight.
 *   ws, ws_bytes  scratch of fm_norm_residual_workspace_bytes, 16-byte aligned,
 *            without preparation; needed if any of these three is wanted, one
 *            for each call that may run at the same time.
 * The column sums are taken in a fixed order: identical bits on every call.
 */
size_t fm_norm_residual_workspace_bytes(int64_t M, int64_t N, int64_t n_gates);

fm_status_t fm_norm_residual_bwd(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt,
                                 int64_t M, int64_t N, const void* d_y, const void* d_out,
                                 const void* out, const void* block, const void* w_post,
                                 const void* w_pre, const void* gate, int64_t n_gates,
                                 float scale, const float* rstd_post, const float* rstd_pre,
                                 void* d_resid, void* d_block, float* d_w_post, float* d_w_pre,
                                 float* d_gate, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * 4-bit weights.  A [K, N] matrix is N * fm_w4_row_bytes(K) packed bytes, with
 *   W[k, n] = (code[k, n] - zero[k / group, n]) * scale[k / group, n],
 * codes 0..15; scales [ceil(K / group), N] in the activations' type; zeros
 * uint8 of the same shape, or NULL: 8 everywhere; group 32, 64 or 128 (the last
 * group of a K may be short).  Column n is a row of fm_w4_row_bytes(K) =
 * 64 * ceil(K / 128) bytes.  Each 64-byte block holds 128 k as 16 little-endian
 * words: word 4 q + j holds k = 32 j + 8 q + 0..7, its nibble p, from the low
 * end, the k offset 2 p for p < 4 and 2 (p - 4) + 1 for p >= 4 (so that one
 * 16-byte load of a lane feeds four matrix instructions).  Codes past K are
 * not used.
 *
 * fm_w4_pack -- packed bytes from codes, uint8 [n_matrices, K, N], values
 * 0..15 (the high four bits are dropped).  Done once when weights are loaded.
 */
size_t fm_w4_row_bytes(int64_t K);

fm_status_t fm_w4_pack(int64_t n_matrices, int64_t K, int64_t N, const uint8_t* codes,
                       void* packed, hipStream_t stream);

/*
 * fm_gemm_w4 -- fm_gemm with a 4-bit B, for few rows (a decode step):
 * C[M, N] = A[M, K] * W[K, N].  The weights are read once for every 48 rows;
 * for hundreds of rows, unpacked 16-bit weights and fm_gemm are faster.
 * C must not overlap A.
 *   ab      FM_F16 or FM_BF16: A and scales;  c  ab or FM_F32.
 *   packed  as above, 16-byte aligned; scales 16-byte aligned.
 * Codes enter the matrix cores exactly; products are summed in fp32 group by
 * group and scaled there: codes as 16 + code, with 16 + zero times the sum of A
 * taken off afterwards, so a result's error is relative to sum |A| (16 + code)
 * scale.  A must be finite, and 31 times the sum of a group's |A| below 2^128; an
 * infinite or NaN A[m, k] makes row m of C NaN or infinite.
 */
fm_status_t fm_gemm_w4(fm_dtype_t ab, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                       int32_t group, const void* A, const void* packed, const void* scales,
                       const uint8_t* zeros, void* C, hipStream_t stream);

/*
 * fm_moe_gather_gemm_w4 -- fm_moe_gather_gemm_act with 4-bit weights, for the
 * few tokens of a decode step: packed, scales and zeros hold n_local
 * [hidden, ffn] matrices.  The other arguments, sorted_pairs, expert_offsets
 * and the rows of H behind them as there; ws is that call's workspace.
 * Experts without a token are not read.
 */
fm_status_t fm_moe_gather_gemm_w4(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                                  int32_t topk, int32_t expert_begin, int32_t n_local,
                                  int32_t group, const void* X, const int32_t* topk_ids,
                                  const void* packed, const void* scales, const uint8_t* zeros,
                                  void* H, int32_t* sorted_pairs, int32_t* expert_offsets,
                                  fm_act_t act, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * fm_moe_gemm_scatter_w4 -- the combine with 4-bit weights, for few tokens:
 *   out[t, :] = add[t, :] + sum over local pairs p = t*topk + k of
 *               topk_weights[p] * (H[row(p), :] * W2[e(p)])
 * summed in the order of k.  packed, scales and zeros hold n_local
 * [ffn, hidden] matrices; H, sorted_pairs and expert_offsets are those of
 * fm_moe_gather_gemm_w4 (or fm_moe_gather_gemm) with the same topk_ids and
 * expert_begin.  Two pairs of a token may name one expert.
 *   add  fp32 [T, hidden] or NULL: 0; it may be out itself (out += ...).
 *   ws, ws_bytes  scratch of fm_moe_w4_workspace_bytes, 16-byte aligned,
 *        without preparation; one for each call that may run at the same time.
 * Deterministic: identical bits on every call.
 */
size_t fm_moe_w4_workspace_bytes(int64_t T, int32_t topk, int64_t hidden);

fm_status_t fm_moe_gemm_scatter_w4(fm_dtype_t dt, int64_t T, int64_t hidden, int64_t ffn,
                                   int32_t topk, int32_t expert_begin, int32_t n_local,
                                   int32_t group, const void* H, const void* packed,
                                   const void* scales, const uint8_t* zeros,
                                   const int32_t* topk_ids, const int32_t* sorted_pairs,
                                   const int32_t* expert_offsets, const float* topk_weights,
                                   const float* add, float* out, void* ws, size_t ws_bytes,
                                   hipStream_t stream);

/*
 * fm_dropout -- y = x * s where an element is kept, 0 where it is dropped (whatever x
 * is there), from a counter-based generator: the mask is a function of seed, offset
 * and place alone and is never stored.  The backward pass is the same call on the
 * gradient.  Element (i, j) has the 16-bit number
 *   half c % 8 of philox4x32_10(counter, key),  r = row_begin + i, c = col_begin + j,
 *   counter = (c / 8, r, low and high word of rng[1] + draw),  key = rng[0],
 * halves counted from the low end of word 0, and is kept if that is below t;
 *   t = (1 - p) * 65536 rounded,   s = 65536 / t.
 * (Philox: Salmon, Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3",
 * 2011.)  A GPU that holds some rows or columns of a tensor draws with row_begin and
 * col_begin what one that holds all of it would.
 *   dt         FM_F16, FM_BF16 or FM_F32.   x, y  [M, N]; y may be x itself.
 *   p          share of dropped elements, 0..1; 0 copies, 1 clears.
 *   rng        device uint64 [2]: seed and offset; read when the kernel runs, so a
 *              captured graph draws anew if the program advances rng[1] between
 *              replays.  8-byte aligned; NULL only with p = 0.
 *   draw       added to the offset (both wrap round): one number for each place of a
 *              program that draws, the same in forward and backward.  Two draws with one
 *              sum share their mask: a program whose places have the numbers 0 .. n - 1
 *              advances rng[1] by n from step to step.
 *   row_begin, col_begin  >= 0; col_begin a multiple of 8; row_begin + M at most
 *              2^32, col_begin + N at most 2^34.
 */
fm_status_t fm_dropout(fm_dtype_t dt, int64_t M, int64_t N, const void* x, float p,
                       const uint64_t* rng, int64_t draw, int64_t row_begin, int64_t col_begin,
                       void* y, hipStream_t stream);

/*
 * fm_layer_norm -- what lies between two products of a dense block's residual stream,
 * in one pass.  For each row
 *   out = resid + dropout(block + bias)
 *   y   = (out - mean) * rstd * w + b     mean, rstd = 1 / sqrt(variance + eps) of out
 * all in fp32 (y from the fp32 value of out), rounded once when stored.  block may be
 * a slice that fm_gemm_rs filled (fp32); y is the 16-bit input of fm_ag_gemm, or the
 * 8-bit one of fm_gemm_i8.
 *   dt         FM_F16 or FM_BF16: y, bias, w and b.
 *   stream_dt  resid and out: dt or FM_F32.   block_dt  block: dt or FM_F32.
 *   M, N       rows and row length; N a multiple of 8, at most 16384.
 *   block      [M, N] or NULL: nothing is added (bias must be NULL and p 0).
 *   resid      [M, N] or NULL: 0.  Not both NULL.
 *   bias       [N] or NULL: 0.
 *   w          [N], or NULL: no norm.  y is NULL if and only if w is.
 *   b          [N] or NULL: 0; only with w.
 *   p, rng, draw, row_begin  as fm_dropout (columns from 0).
 *   out        [M, N] or NULL (not wanted); it may be resid itself.
 *   y_scale    fp32 [M]: y is int8, its rows as fm_quant_i8 makes them of the fp32
 *              values.  NULL: y is in dt.
 *   mean, rstd fp32 [M] or NULL, which the backward needs; only with w.
 */
fm_status_t fm_layer_norm(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                          int64_t N, const void* block, const void* resid, const void* bias,
                          const void* w, const void* b, float p, const uint64_t* rng,
                          int64_t draw, int64_t row_begin, float eps, void* out, void* y,
                          float* y_scale, float* mean, float* rstd, hipStream_t stream);

/*
 * fm_layer_norm_bwd -- gradients of fm_layer_norm.
 *   d_y      [M, N] dt, gradient of y; NULL if and only if w is.
 *   d_out    [M, N] stream_dt, gradient of out from its later uses, or NULL: 0
 *            (without w it is needed).
 *   out      [M, N] stream_dt, and mean, rstd, as the forward stored them; needed with w.
 *   p, rng, draw, row_begin  as in the forward.
 *   d_resid  [M, N] stream_dt or NULL: gradient of resid (of out in total).
 *            It may be d_out itself.
 *   d_block  [M, N] block_dt or NULL.
 *   d_bias, d_w, d_b  fp32 [N], written whole, or NULL; d_w and d_b only with w.
 *   ws, ws_bytes  scratch of fm_layer_norm_workspace_bytes, 16-byte aligned, without
 *            preparation; needed if any of these three is wanted, one for each call
 *            that may run at the same time.
 * The column sums are taken in a fixed order: identical bits on every call.
 */
size_t fm_layer_norm_workspace_bytes(int64_t M, int64_t N);

fm_status_t fm_layer_norm_bwd(fm_dtype_t dt, fm_dtype_t stream_dt, fm_dtype_t block_dt, int64_t M,
                              int64_t N, const void* d_y, const void* d_out, const void* out,
                              const float* mean, const float* rstd, const void* w, float p,
                              const uint64_t* rng, int64_t draw, int64_t row_begin,
                              void* d_resid, void* d_block, float* d_bias, float* d_w,
                              float* d_b, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * 8-bit integers.  fm_quant_i8 -- rows in 8 bits with a scale each: with
 * top = max |x[i, :]|,
 *   scale[i] = top / 127     q[i, j] = 127 x[i, j] / top, rounded to nearest even,
 * so x[i, j] is about q[i, j] * scale[i].  A row whose top is below 2^-100 is held as
 * zeros with scale 0; one that holds a NaN, or whose top is 2^120 or more, as zeros
 * with scale NaN (a row of NaN, not of wrong numbers, in what is made of it).
 * Activations have a row for each token; a weight matrix [N, K] has a row, and so a
 * scale, for each output channel.
 *   dt  FM_F16, FM_BF16 or FM_F32: x [M, N];  q int8 [M, N], not overlapping x;  scale
 *       fp32 [M].  M and N below 2^31.
 */
fm_status_t fm_quant_i8(fm_dtype_t dt, int64_t M, int64_t N, const void* x, int8_t* q,
                        float* scale, hipStream_t stream);

/*
 * fm_gemm_i8 -- product of 8-bit rows:
 *   C[m, n] = act(a_scale[m] * w_scale[n] * sum_k A[m, k] * W[n, k] + bias[n]).
 * The sum is exact (32-bit integers); scales, bias and activation are applied in fp32
 * and the result is rounded once.  a_scale[m] * w_scale[n] is taken first: past 2^128 a value
 * is infinite, or NaN where the sum is 0; below 2^-126 it has fewer bits.
 *   dt       FM_F16 or FM_BF16: bias;  c  dt or FM_F32: C.
 *   A        int8 [M, K] with a_scale fp32 [M];  W  int8 [N, K] (an output channel's
 *            weights in a row) with w_scale fp32 [N].  -128 may occur.
 *   bias     [N] or NULL: 0.   act  fm_act_t.   C  [M, N].
 *   K a multiple of 16, at most 131056 (the sums fit 32 bits); N a multiple of 8; M and
 *   N below 2^22; w_scale 16-byte aligned.  C must not overlap the operands.  A NaN or
 *   infinite scale stays in its row or column, a NaN under every activation.
 */
fm_status_t fm_gemm_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                       const int8_t* A, const float* a_scale, const int8_t* W,
                       const float* w_scale, const void* bias, fm_act_t act, void* C,
                       hipStream_t stream);

/*
 * fm_linear_i8 -- fm_quant_i8 of the rows of X, then fm_gemm_i8: a linear layer with
 * 8-bit weights on 16-bit activations, the same bits as those two calls.
 *   X   [M, K] in dt.   ws, ws_bytes  scratch of fm_linear_i8_workspace_bytes, 16-byte
 *       aligned, without preparation; one for each call that may run at the same time.
 */
size_t fm_linear_i8_workspace_bytes(int64_t M, int64_t K);

fm_status_t fm_linear_i8(fm_dtype_t dt, fm_dtype_t c, int64_t M, int64_t N, int64_t K,
                         const void* X, const int8_t* W, const float* w_scale, const void* bias,
                         fm_act_t act, void* C, void* ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FLUXMI_H */
