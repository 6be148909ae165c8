/*
 * jfa.h -- C ABI of libjfa, jagged FlashAttention forward and backward for
 * GB300 (sm_103a).
 *
 * The operation (jagged FlashAttention pages: the alphasignal news page,
 * section "GEM's sequences do not fit a fixed grid"; the PyTorch-blog summary
 * on arc-codex, first key point): B variable-length sequences are packed
 * back to back, with no padding, and addressed by an offsets array, and
 * FlashAttention runs on them in that form; for every sequence b and head h
 *
 *     O_b = softmax(scale * Q_b K_b^T) V_b,   LSE_b = logsumexp(scale * Q_b K_b^T)
 *
 * row by row, with no mask inside a sequence.  In broadcast mode one dense
 * query block Q [Lq, H, D] attends to every sequence (same page and section:
 * all sequences of a batch share the query block, so their query gradients
 * add up) and the backward sums dQ over the batch.
 *
 * Layouts (all row-major, contiguous):
 *   K, V        bf16 [kv_offsets[B], H, D]
 *   Q           bf16 [q_offsets[B], H, D]            (self mode)
 *               bf16 [Lq, H, D]                      (broadcast mode)
 *   O, dO       bf16 [n_o, H, D], n_o = q_offsets[B] (self) or B*Lq (broadcast, b-major)
 *   LSE         fp32 [H, n_o], natural log of the row sum, scale included;
 *               -inf for rows of a sequence with no keys
 *   dQ          fp32, the shape of Q (broadcast: summed over all sequences)
 *   dK, dV      bf16, the shape of K
 * bf16 is IEEE-754 binary16-brain (8-bit exponent), passed as raw 16-bit
 * words.  Supported: D in {64, 128}; every device pointer 16-byte aligned.
 *
 * Ownership: the caller owns every tensor and the stream.  A plan owns a
 * small device copy of the offsets and of the tile schedule; it must outlive
 * the stream work that uses it.  A plan belongs to the device that was
 * current when it was created: jfa_fwd, jfa_bwd (and its stages) and
 * jfa_plan_device_status return JFA_ERR_INVALID_ARG when another device is
 * current.  jfa_fwd / jfa_bwd allocate nothing and are
 * asynchronous on the given stream (a cudaStream_t passed as void*; NULL is
 * the legacy default stream).
 *
 * Errors: every entry point returns a jfa_status; nothing throws across the
 * ABI.  Argument problems are reported before anything is launched.  Device
 * waits in the kernels are bounded: a wait that runs out records
 * JFA_ERR_DEVICE_TIMEOUT in the plan's device status word, which
 * jfa_plan_device_status reads back.
 */
#ifndef JFA_H
#define JFA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum jfa_status {
  JFA_OK = 0,
  JFA_ERR_INVALID_ARG = 1,    /* null pointer, non-positive size, bad direction ... */
  JFA_ERR_UNSUPPORTED = 2,    /* D not in {64, 128}, no sm_100-family GPU */
  JFA_ERR_BAD_OFFSETS = 3,    /* offsets[0] != 0, decreasing, or total >= 2^31 */
  JFA_ERR_ALIGNMENT = 4,      /* a device pointer is not 16-byte aligned */
  JFA_ERR_WORKSPACE = 5,      /* workspace missing or smaller than jfa_bwd_workspace_bytes */
  JFA_ERR_CUDA = 6,           /* a CUDA runtime call failed */
  JFA_ERR_DEVICE_TIMEOUT = 7, /* a kernel wait ran out (see jfa_plan_device_status) */
  JFA_ERR_PAGES = 8           /* a paged call met bad lengths, pages or slots, or ran out of pages
                                 (see jfa_pager_status) */
} jfa_status;

/* Tile geometry: query rows per forward tile and key rows per backward tile. */
#define JFA_BLOCK_M 128
#define JFA_BLOCK_N 128

typedef struct jfa_plan* jfa_plan_t;

/*
 * Build a plan for one batch shape.
 *   kv_offsets_host  int32 [B+1], host memory: kv_offsets[0] = 0, non-decreasing.
 *   q_offsets_host   int32 [B+1] host offsets of the queries (self mode; may
 *                    equal kv_offsets), or NULL for broadcast mode.
 *   B, H             sequences and heads (B >= 1, H >= 1).
 *   Lq               broadcast mode: rows of the dense Q (>= 0); ignored in self mode.
 *   D                head dimension, 64 or 128.
 *   num_ctas         persistent CTAs per launch; 0 = one per SM of the current device.
 *   stream           stream for the host-to-device upload of offsets and tiles.
 * The tile schedule follows the pages' description: forward tiles
 * (b, h, query block) are sorted by key/value workload and dealt to the CTAs
 * in zigzag (boustrophedon) order (alphasignal page, "Five changes unlocked
 * the gains", item 1); backward tiles (b, h, key block) exist only where the
 * sequence has queries and are dealt round-robin (yuxiaoba note, "Why both
 * static and dynamic balancing help").  On success *out receives the plan.
 * Allocates device memory; the host arrays are not retained.
 */
int jfa_plan_create(const int32_t* kv_offsets_host, const int32_t* q_offsets_host, int B, int H,
                    int Lq, int D, int num_ctas, void* stream, jfa_plan_t* out);

/*
 * Plan flags.
 * Packing of short sequences: in self mode with one offsets array shared by
 * queries and keys (q_offsets equal to kv_offsets element by element), runs
 * of consecutive short sequences whose lengths add up to at most 128 rows
 * (with at least two non-empty ones) share one 128-row tile, masked
 * block-diagonally so every row still sees only its own sequence.  This is
 * the block-diagonal case of the TLX Block Attention page ("One Constraint,
 * Five Eliminations": each query tile meets exactly one key tile), which an
 * unpacked schedule runs at half occupancy when segments are shorter than a
 * tile.  Such a tile is recorded as {b0, h, -nseq, 1}.  Never in broadcast
 * mode or when the offsets differ.  By default a plan packs when that removes
 * at least an eighth of its forward tiles (a pack of n non-empty sequences
 * replaces n tiles by one).
 * JFA_PLAN_PACK_SHORT: pack whenever a run forms.
 * JFA_PLAN_NO_PACK: never pack.  Setting both is JFA_ERR_INVALID_ARG.
 */
#define JFA_PLAN_PACK_SHORT 1u
#define JFA_PLAN_NO_PACK 32u

/*
 * JFA_PLAN_DYNAMIC: tiles are claimed at run time instead of dealt on the
 * host (the pages' dynamic balancing, which works alongside the static order):
 * each schedule lists every tile once in claim order -- the tiles stably
 * sorted by their cost field, largest first -- and the plan's P CTAs take
 * tile blockIdx.x, then the next unclaimed one from a device counter, until
 * none is left.  jfa_plan_tiles / jfa_build_tiles return that list with
 * cta_ptr = {0, T, ..., T} (P + 1 entries: one queue shared by the P CTAs
 * launched).  The
 * counter lives in the plan and is reset on the stream before each launch,
 * so a plan's launches must be stream-ordered.  Combines with
 * JFA_PLAN_PACK_SHORT.
 * JFA_PLAN_DYNAMIC claims the tiles of both passes; JFA_PLAN_STATIC deals
 * both on the host (the two together are invalid).  Without either, the
 * forward is dealt on the host, and the backward is claimed at run time when
 * queries have their own offsets (self mode, where a sequence's key blocks
 * make tiles of very different lengths) and dealt in broadcast mode, where
 * claiming measured slower; jfa_plan_claims reports the choice.
 */
#define JFA_PLAN_DYNAMIC 2u
#define JFA_PLAN_STATIC 128u

/*
 * Where Delta comes from.  When every sequence that has queries has at most
 * 128 keys (one key block: the block-diagonal and other short-sequence
 * cases), each backward tile meets all the keys of its queries and can form
 * Delta_i = sum_j P_ij dP_ij over them itself.  That is the same quantity as
 * sum_d dO_id O_id, because O = P V and dP = dO V^T, so the pre-pass that
 * reads O and dO only for Delta is skipped (the backward then does not read
 * O at all).  The sums cost every tile the same whatever its fill, so by
 * default the tiles form Delta only when they hold at least 96 key rows on
 * average (full tiles, as with JFA_PLAN_PACK_SHORT on 64-token segments).
 * JFA_PLAN_DELTA_PREPASS: always use the pre-pass.
 * JFA_PLAN_DELTA_IN_TILES: let the tiles form Delta whenever they hold all
 *   the keys of their queries, whatever their fill.
 * Setting both is JFA_ERR_INVALID_ARG.
 */
#define JFA_PLAN_DELTA_PREPASS 4u
#define JFA_PLAN_DELTA_IN_TILES 8u

/*
 * JFA_PLAN_FWD_PAIRS: run the forward as CTA pairs where the pair kernel
 * applies (D = 128, static schedule, no packed tiles, num_ctas >= 2).  Two
 * CTAs of a thread-block cluster take the two query blocks of a "pair tile"
 * (b, h, mp) -- query rows [256 mp, 256 mp + 256) of sequence b; a sequence
 * with an odd number of query blocks leaves its last pair tile half empty --
 * and share every K/V block, each loading half of it; one thread issues the
 * pair's tensor-core products, which span both CTAs' query rows (M = 256)
 * and so cost the pair fewer instructions than two single-CTA tiles (the
 * pages' 2-CTA collaborative MMA: alphasignal JFA page, "Five changes
 * unlocked the gains", closing paragraph).  The forward schedule then lists
 * pair tiles {b, h, mp, cost} over P = min(num_ctas / 2, T) pairs.
 * Without the flag a plan runs one CTA per query block: on GB300 that form
 * measures faster on every workload tried (the pair's K/V loads, half per
 * CTA plus the peer's half over the pair, arrive no sooner than a single
 * CTA's whole block, and its query blocks share no K/V through L2).
 */
#define JFA_PLAN_FWD_PAIRS 64u

/*
 * JFA_PLAN_FWD_TWO: run the forward with two query tiles in flight per CTA
 * where that kernel applies (D = 128, static schedule, no packed tiles):
 * each schedule tile {b, h, mp, cost} covers query blocks 2 mp and 2 mp + 1
 * of sequence b -- the list jfa_build_tiles dir 2 gives, over num_ctas CTAs
 * -- and the CTA alternates between them, so one tile's tensor-core products
 * run while the other tile's softmax works (the pages' two query tiles per
 * CTA: alphasignal JFA page, "Specialized warps keep tensor cores busy").
 * A sequence with an odd number of query blocks leaves its last tile half
 * empty.  By default a plan runs this form where it applies, its tiles
 * hold at least 3 key blocks on average with at most a quarter of them half
 * empty, and there are at least four of them per CTA (measured faster there,
 * slower on short tiles and on few tiles per CTA); JFA_PLAN_FWD_TWO
 * asks for it wherever it applies, JFA_PLAN_FWD_ONE never.  At most one of
 * JFA_PLAN_FWD_PAIRS, JFA_PLAN_FWD_TWO and JFA_PLAN_FWD_ONE (invalid
 * together).
 */
#define JFA_PLAN_FWD_TWO 256u
#define JFA_PLAN_FWD_ONE 512u

/* jfa_plan_create with flags (0 = the schedule described above). */
int jfa_plan_create_ex(const int32_t* kv_offsets_host, const int32_t* q_offsets_host, int B, int H,
                       int Lq, int D, int num_ctas, unsigned flags, void* stream, jfa_plan_t* out);

/* Release a plan (synchronises the device first so in-flight work finishes). */
int jfa_plan_destroy(jfa_plan_t plan);

/*
 * Copy a plan's tile schedule to host memory.  dir: 0 forward (the schedule
 * the plan launches: over tiles of two query blocks when it runs CTA pairs or
 * two tiles per CTA, see jfa_plan_forward_form), 1 backward.
 * tiles_host receives T records of four int32 {b, h, block, cost} grouped by
 * CTA (or pair), cta_ptr_host receives P+1 CSR offsets (P = min(num_ctas, T),
 * or the number of pairs).  Either
 * buffer may be NULL to query only *T and *P.  Buffers must hold 4*T and P+1
 * int32.
 */
int jfa_plan_tiles(jfa_plan_t plan, int dir, int32_t* tiles_host, int32_t* cta_ptr_host, int* T,
                   int* P);

/* *fwd / *bwd = 1 when that pass's tiles are claimed at run time (JFA_PLAN_DYNAMIC
 * and the default rule given with it), 0 when they are dealt on the host.
 * Either pointer may be NULL. */
int jfa_plan_claims(jfa_plan_t plan, int* fwd, int* bwd);

/* *form = 0 when the plan's forward runs one query tile per CTA, 1 as CTA
 * pairs (JFA_PLAN_FWD_PAIRS), 2 with two query tiles per CTA (JFA_PLAN_FWD_TWO). */
int jfa_plan_forward_form(jfa_plan_t plan, int* form);

/* *pairs = 1 when the plan's forward runs as CTA pairs (JFA_PLAN_FWD_PAIRS), else 0. */
int jfa_plan_forward_pairs(jfa_plan_t plan, int* pairs);

/*
 * Host-only schedule builder (no GPU needed): the same lists a plan created
 * with the same flags holds.  dir: 0 forward (one CTA per query block), 1
 * backward, 2 forward over pair tiles (num_ctas then counts CTA pairs).
 * q_offsets_host == NULL means broadcast with Lq rows.  Call once with
 * tiles_out == NULL to learn *T and *P, then with buffers of 4*T and P+1
 * int32.
 */
int jfa_build_tiles(const int32_t* kv_offsets_host, const int32_t* q_offsets_host, int B, int H,
                    int Lq, int num_ctas, int dir, unsigned flags, int32_t* tiles_out,
                    int32_t* cta_ptr_out, int* T, int* P);

/*
 * Host-only (no GPU needed): the schedule choices jfa_plan_create_ex makes
 * for these arguments on a device of num_ctas SMs (num_ctas >= 1 here):
 * *fwd_form as jfa_plan_forward_form, *fwd_claims / *bwd_claims as
 * jfa_plan_claims, *packed = 1 when short sequences are packed into shared
 * tiles (JFA_PLAN_PACK_SHORT's rule).  Any output pointer may be NULL.
 * Errors as jfa_plan_create_ex (offsets, sizes, conflicting flags).
 */
int jfa_plan_choices(const int32_t* kv_offsets_host, const int32_t* q_offsets_host, int B, int H,
                     int Lq, int D, int num_ctas, unsigned flags, int* fwd_form, int* fwd_claims,
                     int* bwd_claims, int* packed);

/*
 * Host-only (no GPU needed): *in_tiles = 1 when a plan created from these
 * offsets and flags has its backward tiles form Delta (the rule given with
 * JFA_PLAN_DELTA_PREPASS), 0 when the pre-pass forms it.  With 1, jfa_bwd
 * does not read `out`; jfa_bwd_noalloc follows the flags-0 answer.  Errors as
 * jfa_plan_create_ex (offsets, conflicting Delta flags).
 */
int jfa_delta_in_tiles(const int32_t* kv_offsets_host, const int32_t* q_offsets_host, int B,
                       int Lq, unsigned flags, int* in_tiles);

/*
 * Forward: out = softmax(scale Q K^T) V per sequence and head, lse as above.
 * q, k, v, out: bf16 device tensors in the layouts above; lse: fp32 device.
 * Rows of sequences without keys get O = 0 and LSE = -inf.
 */
int jfa_fwd(jfa_plan_t plan, const void* q, const void* k, const void* v, float scale, void* out,
            float* lse, void* stream);

/* Bytes of device workspace jfa_bwd needs (the fp32 row sums Delta = rowsum(dO * O)). */
size_t jfa_bwd_workspace_bytes(jfa_plan_t plan);

/*
 * Backward of jfa_fwd.  Inputs q, k, v, out (the forward's O), dout (dO), lse
 * (the forward's LSE) and the forward's scale.  Outputs dq (fp32, overwritten -- the library clears it
 * on the stream), dk and dv (bf16).  workspace: device memory of at least
 * jfa_bwd_workspace_bytes(plan) bytes, 16-byte aligned.  The backward first
 * forms Delta_i = sum_d dO_id O_id (the row sum the TLX Block Attention page
 * calls the "Di" preprocessing, "One Constraint, Five Eliminations"), then
 * runs the key/value-stationary pass that produces dK, dV and reduce-adds dQ.
 * Where every tile holds all the keys of its queries, the main pass may form
 * Delta itself instead (see JFA_PLAN_DELTA_PREPASS); the workspace is then
 * not written, but its size and alignment rules stay the same.
 */
int jfa_bwd(jfa_plan_t plan, const void* q, const void* k, const void* v, const void* out,
            const void* dout, const float* lse, float scale, float* dq, void* dk, void* dv,
            void* workspace, size_t workspace_bytes, void* stream);

/*
 * The two stages jfa_bwd runs, for callers that schedule them separately
 * (same arguments and rules as jfa_bwd).
 * jfa_bwd_preprocess: Delta (into workspace) from out and dout -- skipped when
 *   the main pass forms Delta itself (see JFA_PLAN_DELTA_PREPASS) --, clears the dq
 *   rows the main pass reduce-adds into or never writes (all of them in
 *   broadcast mode; with query offsets, those of sequences with no key or
 *   more than one key block -- a sequence with one key block, or in a packed
 *   tile, has its dQ rows stored outright by its one tile), and zeroes dk / dv
 *   rows of sequences with keys but no queries.
 * jfa_bwd_main: the key/value-stationary pass; needs the workspace written by
 *   jfa_bwd_preprocess (stream order) and the dq rows it cleared.
 */
int jfa_bwd_preprocess(jfa_plan_t plan, const void* out, const void* dout, float* dq, void* dk,
                       void* dv, void* workspace, size_t workspace_bytes, void* stream);
int jfa_bwd_main(jfa_plan_t plan, const void* q, const void* k, const void* v, const void* dout,
                 const float* lse, float scale, float* dq, void* dk, void* dv,
                 const void* workspace, size_t workspace_bytes, void* stream);

/*
 * Read the plan's device status word (synchronises `stream`), then clear it.
 * Returns JFA_ERR_DEVICE_TIMEOUT when a kernel recorded a wait that ran out,
 * JFA_OK otherwise; *raw (optional) receives the raw word.
 */
int jfa_plan_device_status(jfa_plan_t plan, void* stream, int* raw);

/*
 * Backward for callers that cannot allocate device memory: code that runs
 * inside a framework whose caching or pool allocator owns all device memory
 * (a stray cudaMalloc there fragments or oversubscribes the pool, and
 * cudaFree synchronises the device), and embedded or serving runtimes that
 * are handed a fixed budget of pre-allocated buffers and may not grow it.
 * There is no counterpart of this entry point on the jagged FlashAttention
 * pages; it computes exactly what jfa_bwd computes (same inputs, outputs,
 * layouts and tolerances) but needs neither a plan nor a workspace.
 *
 * Arguments are those of jfa_plan_create (host offsets, B, H, Lq, D) followed
 * by those of jfa_bwd without workspace; device_status is an optional device
 * int the kernels set when a wait runs out (NULL: not reported).
 *
 * Scratch: the schedule, the device copy of the offsets and the Delta row
 * sums live in one file-scope static __device__ array of
 * JFA_NOALLOC_SCRATCH_BYTES, which every GPU that loads this library holds
 * until the process exits.  A problem whose scratch (about 4 * H * n_o bytes
 * of Delta plus 16 bytes per backward tile; no Delta where the tiles form it,
 * under the default rule given with JFA_PLAN_DELTA_PREPASS) does not fit is
 * rejected with
 * JFA_ERR_WORKSPACE before anything is launched, as is (JFA_ERR_UNSUPPORTED)
 * any problem jfa_plan_create would refuse.  The call allocates no device
 * memory and calls no allocating library routine.  It uploads the schedule
 * and offsets with cudaMemcpyAsync from a host buffer that lives only for
 * the call (pageable memory), so the call returns once that copy has been
 * taken from the host buffer, and the call cannot be captured into a CUDA
 * graph (a replay would read that buffer after the call has returned).
 *
 * The first call on a device resolves the array's device address
 * (cudaGetSymbolAddress, with that device current).  All calls share the one array and each call
 * rewrites what it needs (nothing is assumed to start at zero), so calls
 * that overlap on the GPU -- different streams, or different host threads
 * without ordering -- race; issue them on one stream or order them.
 */
#define JFA_NOALLOC_SCRATCH_BYTES (32u << 20)
int jfa_bwd_noalloc(const int32_t* kv_offsets_host, const int32_t* q_offsets_host, int B, int H,
                    int Lq, int D, const void* q, const void* k, const void* v, const void* out,
                    const void* dout, const float* lse, float scale, float* dq, void* dk, void* dv,
                    int* device_status, void* stream);

/*
 * Test of the kernels' failure path (no counterpart in the pages; it exists
 * so that the timeout handling of the real kernels can be exercised on a GPU
 * without a fault).  Sets, for the plan's later launches, a limit of
 * limit_us microseconds on every device wait (0: the normal 2 s; at most
 * 2,000,000) and, with skip != 0, has one softmax warp of CTA 0 withhold one
 * arrival so that a wait of the MMA issuer runs out:
 *   skip = 1  jfa_fwd: the arrival on the first P block of CTA 0's first tile
 *   skip = 2  jfa_bwd: the arrival on the first dS^T block of CTA 0
 *   skip = 0  nothing withheld (normal operation)
 * The wait that runs out raises the CTA's abort flag: every role leaves its
 * loop, the TMA producer and the MMA issuer wait (bounded) for their work in
 * flight, and the TMEM is freed before the CTA exits, so the context stays
 * usable; jfa_plan_device_status then reports JFA_ERR_DEVICE_TIMEOUT, and the
 * outputs of that launch are undefined.  Not for production use: nothing in
 * the library or its benchmark sets it.  Errors: JFA_ERR_INVALID_ARG.
 */
int jfa_plan_selftest(jfa_plan_t plan, int skip, unsigned limit_us);

/*
 * Self-test of the failure path (no counterpart in the pages; it exists so
 * the timeout handling every kernel relies on can be exercised on a GPU
 * without a fault).  Launches one CTA whose waiting thread runs the kernels'
 * bounded mbarrier wait on a barrier nothing arrives on, with the limit
 * shortened to limit_us microseconds (1 .. 2,000,000), and synchronises the
 * stream.  Expected result: JFA_ERR_DEVICE_TIMEOUT, with the wait's measured
 * duration in *waited_ns (may be NULL); the kernel returns normally, so the
 * context stays usable.  JFA_OK would mean the wait completed (it cannot);
 * JFA_ERR_CUDA reports a failed launch.  The status word is one static device
 * variable: calls on different streams race.
 */
int jfa_selftest_wait_timeout(unsigned limit_us, unsigned long long* waited_ns, void* stream);

/*
 * Diagnostic: what one tensor-core product costs on this GPU.  One CTA issues
 * `count` (a multiple of 8, up to 2^20) tcgen05.mma products of one form back
 * to back into one TMEM accumulator (bf16 operands, fp32 accumulation, K = 16
 * per product, the operand descriptors the attention kernels use) and times
 * them in SM clock cycles: *cycles to the completion of a final commit,
 * *issue_cycles (optional) the time the issuing thread spends handing them
 * over.  group = 0: one run of `count` products; group > 0 (a multiple of 8
 * dividing count): after every `group` products the thread commits and waits
 * for them to complete before the next group, the dependent chain of the
 * kernels (a group's results feed the work the next group needs).
 * form: 0 M = 128, N = 128 with A and B in shared memory, both K-major (the
 * forward's QK^T, the backward's S^T and dP^T), 1 M = 128, N = 256, 2 M = 128,
 * N = 128 with A in TMEM, 3 M = 128, N = 64, 4 as 0 with B MN-major (the
 * backward's dK), 5 as 0 with A and B MN-major (the backward's dQ), 6 as 2
 * with B MN-major (the forward's PV, the backward's dV).  Synchronises the
 * stream.  Errors: JFA_ERR_INVALID_ARG,
 * JFA_ERR_CUDA, JFA_ERR_DEVICE_TIMEOUT (the commit did not arrive within the
 * kernels' wait limit).
 */
int jfa_selftest_mma_cycles(int form, int count, int group, unsigned long long* cycles,
                            unsigned long long* issue_cycles, void* stream);

/*
 * Plan-free forward and backward: the tensors, the host offsets and the sizes
 * in one call, as a framework op calls attention, with no plan handle and no
 * workspace.  Arguments mean what they mean for jfa_plan_create (kv_offsets
 * and q_offsets on the host, q_offsets NULL for broadcast mode with Lq query
 * rows), jfa_fwd and jfa_bwd (device tensors in the same layouts, 16-byte
 * aligned; dq fp32, overwritten).
 *
 * The library keeps a plan for each distinct (device, B, H, Lq, D, offsets)
 * it has seen, up to 8, releasing the least recently used one when a ninth
 * arrives; each cached plan owns the backward's workspace.  The first call
 * with new offsets builds the plan (host schedule, one device allocation and
 * an upload synchronised on `stream`), the first backward allocates the
 * workspace; later calls with the same offsets allocate nothing and are
 * asynchronous.  Releasing a plan frees device memory, which synchronises the
 * device.  Calls are serialised by a lock; backward calls with the same
 * offsets that overlap on the GPU (different streams, no ordering) share the
 * workspace and race: order them.
 *
 * Errors: the plan-creation codes (checked before any CUDA call where they
 * need no device), then those of jfa_fwd / jfa_bwd.  A wait that ran out is
 * recorded in the cached plan; jfa_simple_device_status reports it.
 */
int jfa_fwd_simple(const void* q, const void* k, const void* v, const int32_t* kv_offsets_host,
                   const int32_t* q_offsets_host, int B, int H, int Lq, int D, float scale,
                   void* out, float* lse, void* stream);
int jfa_bwd_simple(const void* q, const void* k, const void* v, const int32_t* kv_offsets_host,
                   const int32_t* q_offsets_host, int B, int H, int Lq, int D, float scale,
                   const void* out, const void* dout, const float* lse, float* dq, void* dk,
                   void* dv, void* stream);

/* Device status of every cached plan of the current device (synchronises
 * `stream`, then clears the words): JFA_ERR_DEVICE_TIMEOUT when any recorded
 * a wait that ran out; *raw (optional) receives the words or-ed together. */
int jfa_simple_device_status(void* stream, int* raw);

/* Release every cached plan and workspace (synchronises the device). */
int jfa_simple_release(void);

/*
 * Rotary positions.  A pair of values (a, b) of a head becomes
 *     (a cos phi - b sin phi, b cos phi + a sin phi),
 *     phi = positions[row][axis[i]] * inv_freq[i]
 * for pair i = 0 .. pairs-1, with one position per row and axis (time, height
 * and width of a patch, say; axis[i] in 0 .. 3).  Pair i is (x[i], x[i + pairs]),
 * or (x[2i], x[2i+1]) with JFA_ROTARY_INTERLEAVED; the D - 2*pairs values
 * behind are copied.  D in {64, 128}; pairs a multiple of 8 with 2*pairs <= D.
 *
 * Angles are kept as turns in 64-bit fixed point: inv_freq[i] / (2 pi) is
 * rounded once to a multiple of 2^-64 when the handle is made, its product
 * with an int32 position wraps at whole turns without loss, and its upper 32
 * bits, rounded to fp32, go to the sine and cosine.  The angle that they see is
 * so off by about 2^-26 turns (9.5e-8) at most, at any position.  inv_freq must be
 * finite and below 2^31 in magnitude.
 *
 * The handle holds no device memory: it serves every device and stream, and
 * any number of calls at once.
 */
typedef struct jfa_rotary* jfa_rotary_t;
#define JFA_ROTARY_INTERLEAVED 1u
int jfa_rotary_create(const double* inv_freq_host, const int32_t* axis_host, int pairs, int D,
                      unsigned flags, jfa_rotary_t* out);
int jfa_rotary_destroy(jfa_rotary_t rotary);

/* Host-only: the 64-bit turn fractions a handle made from inv_freq holds. */
int jfa_rotary_turns(const double* inv_freq_host, int pairs, uint64_t* turns_out);

/*
 * Rotate up to two tensors of `rows` rows by the same positions in one launch
 * (x and y: q and k, or their gradients).  x is [rows, x_heads, D] with
 * x_row elements from row to row, heads contiguous; x_out has the same shape
 * and type, its rows x_out_row elements apart.  x_out may be x with the same
 * row distance (in place); otherwise outputs overlap no input.  y == NULL
 * with y_heads 0: one tensor.  Rows are at least heads * D elements apart and
 * a multiple of 16 bytes; tensors are 16-byte aligned.
 * positions: device int32; the position of row r on axis a is
 * positions[r * pos_row + a * pos_axis] (pos_axis 0: one position for every axis).
 * flags: JFA_ROTATE_INVERSE rotates by -phi, which is the gradient of the
 * rotation; JFA_ROTATE_X_FP32 / JFA_ROTATE_Y_FP32: that tensor is fp32 (as
 * jfa_bwd's dq is), otherwise bf16.  Sums are formed in fp32 and rounded once.
 */
#define JFA_ROTATE_INVERSE 1u
#define JFA_ROTATE_X_FP32 2u
#define JFA_ROTATE_Y_FP32 4u
int jfa_rotate(jfa_rotary_t rotary, const int32_t* positions, int64_t pos_row, int64_t pos_axis,
               int64_t rows, unsigned flags, const void* x, int64_t x_row, void* x_out,
               int64_t x_out_row, int x_heads, const void* y, int64_t y_row, void* y_out,
               int64_t y_out_row, int y_heads, void* stream);

/*
 * A paged key/value cache: the rows of K and V live in num_pages pages of
 * page_size rows, [num_pages, page_size, Hkv, D] bf16 (any strides, below),
 * and a request's row t is row t % page_size of page table[b][t / page_size].
 * Row t of page p is also called slot p * page_size + t.  H query heads share
 * Hkv key/value heads: query head h reads key/value head h / (H / Hkv).
 *
 * The caller owns the pages, tables, lengths and the list of free pages, all
 * in device memory, and the pager's block: device memory of at least
 * jfa_pager_block_bytes bytes, 256-byte aligned, which holds the status word
 * and the workspace in which the parts of a split row are joined.  Creating
 * the pager clears part of it on `stream`; it belongs to the pager until that
 * is destroyed and its launches and graphs are done.  A pager belongs to the
 * device that was current when it was created; calls with another device
 * current return JFA_ERR_INVALID_ARG.  Its launches must be stream-ordered,
 * replays of captured graphs among them: use one pager for each stream that
 * decodes at the same time.  Nothing here allocates device memory; calls are
 * asynchronous and may be captured.
 *
 * What only the device can see -- lengths, table entries, slots -- is checked
 * there: nothing outside the given tensors is read or written, the offending
 * request, page or row is left out as each call says, and a bit is set in the
 * status word (jfa_pager_status).
 *
 *   max_seqs    requests of one call, at most 16384; a call of tables or decode has
 *               at least one (B = 0 is JFA_ERR_INVALID_ARG; no rows are fine)
 *   max_pages   columns of the table; (max_pages + 1) * page_size < 2^31
 *   num_pages   pages of the cache; (num_pages + 1) * page_size < 2^31
 *   page_size   rows of a page, any number >= 1
 *   H, Hkv, D   heads (H a multiple of Hkv) and head dimension (64 or 128)
 */
typedef struct jfa_pager* jfa_pager_t;
#define JFA_PAGER_MAX_SEQS 16384
#define JFA_PAGER_NO_PAGES 1   /* status: a request found no free page */
#define JFA_PAGER_BAD_LENGTH 2 /* status: a length, or its change, outside the table's or the rows' bounds */
#define JFA_PAGER_BAD_PAGE 4   /* status: a page, slot or free count outside the cache */
size_t jfa_pager_block_bytes(int H, int Hkv, int D); /* on the current device; 0: unsupported */
int jfa_pager_create(int max_seqs, int max_pages, int64_t num_pages, int page_size, int H, int Hkv,
                     int D, void* block, size_t block_bytes, void* stream, jfa_pager_t* out);
/* Release a pager (its block stays the caller's). */
int jfa_pager_destroy(jfa_pager_t pager);
/* Read the status word (synchronises `stream`), then clear it: JFA_ERR_PAGES
 * when a bit was set; *raw (optional) receives the bits. */
int jfa_pager_status(jfa_pager_t pager, void* stream, int* raw);

/*
 * Block tables and slots from request lengths: request b of B goes from
 * lens[b] to lens[b] + delta[b] rows.  delta > 0 appends that many new rows,
 * delta < 0 drops the last ones (-lens[b]: the request is done).
 *
 * Pages that shrinking requests no longer reach are put on the free list
 * first -- in the order of the requests, and within one by their place in the
 * table, at free_list[n_free], free_list[n_free + 1] ... -- then the growing
 * requests take what they need from its end, in the order of the requests and
 * of their places.  A request of which the free list cannot serve all pages
 * is left as it was, and so are the growing ones behind it that need a page
 * (JFA_PAGER_NO_PAGES).  A request whose length or new length is negative or
 * beyond max_pages * page_size, or whose new rows do not fit into `rows`, is
 * left as it was (JFA_PAGER_BAD_LENGTH).  A count of free pages that is
 * negative or, with the pages given back, above num_pages leaves everything
 * as it was (JFA_PAGER_BAD_PAGE).
 *
 *   lens, delta   int32 [B]
 *   lens_out      int32 [B], the new lengths; may be lens
 *   table         int32 [B, max_pages], its rows table_row apart: entries of
 *                 new pages are written, all others left as they were
 *   free_list     int32 [num_pages]; n_free, n_free_out: int32 [1], may be equal
 *   slots         int32 [rows]: the slot of each new row, requests one after
 *                 the other; -1 for rows of a request left as it was, for rows
 *                 on a page outside the cache (JFA_PAGER_BAD_PAGE) and for
 *                 rows behind the last request's
 *   positions     int32 [rows]: lens[b] + i for the i-th new row; 0 behind
 *   row_offsets   int32 [B + 1]: the first new row of each request (delta > 0
 *                 counts whether the request was left as it was or not)
 * A page belongs to one request: giving back a page that another table shares
 * puts it onto the free list twice.  `rows` is the capacity of slots and
 * positions.  Outputs overlap neither one another nor an input, but as said.  A
 * call whose lens_out and n_free_out are not its lens and n_free can be repeated
 * with the same result.
 */
int jfa_paged_tables(jfa_pager_t pager, int B, const int32_t* lens, const int32_t* delta,
                     int32_t* lens_out, int32_t* table, int64_t table_row, int32_t* free_list,
                     const int32_t* n_free, int32_t* n_free_out, int64_t rows, int32_t* slots,
                     int32_t* positions, int32_t* row_offsets, void* stream);

/* Distances, in elements, of a cache's pages, rows and heads (D contiguous),
 * the same for K and V; multiples of 8, rows less than 2^32 apart. */
typedef struct jfa_pages {
  void* k;
  void* v;
  int64_t page, row, head;
} jfa_pages;

/*
 * Write new rows into the cache: k, v bf16 [rows, Hkv, D] (rows k_row / v_row
 * elements apart, heads contiguous) go to slots[r]; rows with a negative slot
 * are left out, and so are those with a slot outside the cache
 * (JFA_PAGER_BAD_PAGE).  Slots of one call must be distinct, as
 * jfa_paged_tables makes them.  With a rotary handle the keys are rotated on
 * the way by positions (as for jfa_rotate), and so is q [rows, H, D] into
 * q_out when q is given (every row, also those without a slot; q_out may be q
 * with the same row distance).  Otherwise nothing that is written -- the slots'
 * rows, q_out -- overlaps an input.  rotary == NULL: positions, q and q_out are NULL.
 */
int jfa_paged_append(jfa_pager_t pager, int64_t rows, const void* k, int64_t k_row, const void* v,
                     int64_t v_row, const int32_t* slots, const jfa_pages* pages,
                     jfa_rotary_t rotary, const int32_t* positions, int64_t pos_row,
                     int64_t pos_axis, const void* q, int64_t q_row, void* q_out, int64_t q_out_row,
                     void* stream);

/*
 * Attention of one new token per request over its cache:
 *     out[b][h] = softmax(scale * q[b][h] K_b^T) V_b,  lse[h][b] = logsumexp
 * over rows 0 .. lens[b]-1 of request b.  scale is below 2^127 in magnitude (else
 * JFA_ERR_INVALID_ARG), and so are scores: one of -2^127 or less may count as
 * -infinity.  q bf16 [B, H, D] (rows q_row
 * elements apart, heads contiguous), out bf16 [B, H, D], lse fp32 [H, B]
 * (natural log, scale included, as jfa_fwd's); outputs overlap no input (an out
 * that overlaps q is JFA_ERR_INVALID_ARG).  lens[b] = 0: out 0, lse -inf;
 * so too for a length outside 0 .. max_pages * page_size
 * (JFA_PAGER_BAD_LENGTH).  Rows on a page outside the cache are left out
 * (JFA_PAGER_BAD_PAGE).  Rows of a page behind lens[b] may hold anything, NaN
 * and infinities included; an infinite value of V in a counted row makes out
 * infinite, as any weight above 2^-126 of the largest does.  Scores, softmax
 * statistics and sums are fp32; a weight enters the product with V as the sum
 * of two bf16 values, 16 bits in all.  Results are the same, bit for bit, from
 * call to call on the same arguments.
 */
int jfa_paged_decode(jfa_pager_t pager, int B, const void* q, int64_t q_row, const jfa_pages* pages,
                     const int32_t* table, int64_t table_row, const int32_t* lens, float scale,
                     void* out, float* lse, void* stream);

/* Human-readable text of a status code (static storage). */
const char* jfa_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* JFA_H */
