// Declarations of the operators between the q/k/v and the output projection
// and behind the vocabulary projection: the cache append with head norms and
// rotation, attention of drafted tokens over a paged cache, logit penalties.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "operators.h"

namespace w4k {

// Every launch here but the rotation table's is a programmatic dependent of the kernel before it: the kernels touch no memory
// before their dependency wait (the joining launch of the attention reads what its first launch has waited for), so that is legal
// behind anything.

constexpr int T_I8 = 3;                         // W4_I8: a cache of INT8 codes

// One layer's paged cache and the rows of a call (w4_kv_cache, w4_kv_batch).
struct KvView {
    void* k;                  // [pages][Hkv][page][D]
    void* v;
    float* ks;                // [pages][Hkv][page] scales of INT8 codes, or null
    float* vs;
    int type;
    int pages, page, lg;      // lg: log2(page)
    int Hkv, D;
};
struct BatchView {
    const int* table;         // [B][max_pages]
    const int* ctx;           // [B]
    const int* q_start;       // [B + 1]
    int B, max_pages, max_tokens;
};

// ------------------------------------------------ cache append (kv_append.cu)
constexpr int kKaThreads = 128;
struct AppendArgs {
    KvView c;
    BatchView b;
    const void* x;            // [T] rows of ld values: q heads, k heads, v heads
    long long ld;
    int T, Hq;
    const float* turns;       // [positions][rot / 2][2], or null (rot 0)
    int positions, rot, interleaved;
    const int* pos;           // [T], or null: a row's place in the cache
    const float* q_norm;      // [D] or null
    const float* k_norm;
    float eps;
    void* q;                  // [T][Hq][D]
    int qtype;
    int per;                  // loads of heads to a warp (set by the launch)
};
cudaError_t launch_kv_append(AppendArgs& a, int xtype, cudaStream_t s);
cudaError_t launch_kv_values(const KvView& c, bool values, float* out, cudaStream_t s);
cudaError_t launch_rope_table(const double* inv_freq, double factor, double scale, int positions, int half, float* turns,
                              cudaStream_t s);

// ---------------------------------------------- tree attention (attn_tree.cu)
constexpr int kAtUnit = 16;                     // cached tokens of a unit of work
constexpr int kAtRows = 16;                     // query rows of a tile: (token, head of the group)
constexpr int kAtTcUnit = 64;                   // the same of the tensor-core kernel (attn_tc.cu)
constexpr int kAtTcRows = 128;
constexpr int kAtMaxSeq = 1024;
constexpr int kAtMaxTok = 64;                   // drafted tokens of a sequence: the bits of a mask
constexpr int kAtMaxBlocks = 160;
struct AttnArgs {
    CUtensorMap kmap, vmap;
    KvView c;
    BatchView b;
    const void* q;            // [T][Hq][D] of 16 bits
    const unsigned long long* mask;   // [T] or null
    float scale;              // times log2(e)
    int T, Hq, G;             // G = Hq / Hkv
    void* y;                  // [T][Hq][D] of ytype
    int ytype;
    long long units;          // of work, at most (by the table's width)
    int blocks, least, extra; // of the first launch: blocks, units of one at least, units that a second piece is worth
    int* head;                // workspace: B + 1 prefix sums of units (more than 32 sequences)
    float* part;              // workspace: two partial results per block
    int part_rows;            // rows of one
    float* kept;              // workspace of the tensor-core kernel: a block's rows of D
    unsigned* err;
};
__host__ __device__ inline size_t attn_head_bytes(int B) { return (4 * (static_cast<size_t>(B) + 1) + 127) / 128 * 128; }
// A partial result: running maxima, sums, and rows of D.
__host__ __device__ inline size_t attn_part_floats(int rows, int D) { return static_cast<size_t>(rows) * (D + 2); }
cudaError_t launch_attn_tree(AttnArgs& a, int qtype, int sms, cudaStream_t s);
cudaError_t launch_attn_tc(AttnArgs& a, int qtype, int sms, cudaStream_t s);
// Joins the partial results of either kernel (tiles of `rows` rows, units of `unit` tokens).
cudaError_t launch_attn_join(const AttnArgs& a, int rows, int unit, cudaStream_t s);
cudaError_t encode_kv_map(CUtensorMap* map, const AttnArgs& a, const void* base, int box_bytes, int box_rows);

// ------------------------------------------------------ logits (logits.cu)
constexpr int kLgThreads = 256;
constexpr int kLgMaxBias = 1024;
struct LogitArgs {
    const void* x;            // [R] rows of ld values
    void* y;                  // [R] rows of ldy values
    long long ld, ldy;
    int R, V, S;
    const int* ids;           // [S][cap] prompt and generated tokens, or null
    const int* length;        // [S]
    const int* prompt;        // [S]
    int cap;
    const float* rep;         // [S] each, or null
    const float* freq;
    const float* pres;
    const int* bias_ids;      // [S][nb], or null
    const float* bias;        // [S][nb]
    int nb;
    const int* row_start;     // [S + 1], or null: row r is sequence r's
    const int* drafts;        // [R], or null
    const unsigned long long* mask;   // [R], or null
    const unsigned* allowed;  // [R][ceil(V / 32)], or null
    int slices;               // blocks of a copied row (set by the launch)
    int vec;                  // 16-byte words of x are such words of y
};
cudaError_t launch_logits(LogitArgs& a, int type, cudaStream_t s);

// -------------------------------------------------------- device helpers
#ifdef __CUDACC__
// The sequence of a row, by the whole warp: the number of starts behind the
// first that are not above it (B: behind the last sequence).
__device__ __forceinline__ int row_sequence(const int* start, int B, int row, int lane)
{
    int n = 0;
    for (int j = lane; j < B; j += 32) n += __ldg(start + j + 1) <= row;
    return __reduce_add_sync(0xffffffffu, n);
}
#endif

}  // namespace w4k
