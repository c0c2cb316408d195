// regtile_f8_api.hip -- the C ABI's entry points for 8-bit float matrices and for a mixture of experts:
// argument checks (before any HIP call) and the launches.
#include "regtile.h"

#include "f8_common.h"
#include "regtile_internal.h"

namespace {
using regtile::F8Convert;
using regtile::F8Problem;

constexpr int64_t INT_LIMIT = 0x7FFFFFFFll;

bool bad_dtype(int d) { return d != REGTILE_MX_F32 && d != REGTILE_MX_BF16 && d != REGTILE_MX_F16; }
bool misaligned(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == REGTILE_MX_F32 ? 3u : 1u)) != 0; }
bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }  // 32-bit numbers

// A described matrix (or stack of at least `stack`) whose elements are used if `used`
bool bad_matrix(const regtile_f8_matrix *m, bool used, int stack) {
    if (m == nullptr || m->rows < 0 || m->cols < 0 || m->stack < stack) return true;
    if (m->type != REGTILE_F8_E4M3 && m->type != REGTILE_F8_E5M2) return true;
    if (m->block_rows != 1 && m->block_rows != regtile::f8::BLOCK) return true;
    if (m->ld < m->cols || m->ld > INT_LIMIT) return true;
    if (m->scale_row < 0 || m->scale_col < 0 || m->codes_stack < 0 || m->scales_stack < 0) return true;
    if (misaligned(m->scales)) return true;
    return used && m->rows > 0 && m->cols > 0 && (m->codes == nullptr || m->scales == nullptr);
}

// op(m)'s rows along an output dimension, its blocks along k
regtile::F8Operand operand(const regtile_f8_matrix *m, bool rows_are_k) {
    regtile::F8Operand o;
    o.q = m->codes;
    o.s = m->scales;
    o.type = m->type;
    o.shift = m->block_rows == 1 ? 0 : 7;
    o.row = rows_are_k ? 1 : m->ld;
    o.step = rows_are_k ? m->ld : 1;
    o.s_row = rows_are_k ? m->scale_col : m->scale_row;
    o.s_col = rows_are_k ? m->scale_row : m->scale_col;
    return o;
}

bool bad_rows(const regtile_expert_rows *r) {
    if (r == nullptr || r->tokens < 0 || r->k < 1 || r->experts < 1 || r->align < 1) return true;
    // (the size of what passes 2^31 - 1 is -1: a caller may have stored it)
    if (r->rows < 0 || r->rows != regtile_expert_rows_size(r->tokens, r->k, r->experts, r->align)) return true;
    if (r->offsets == nullptr || r->counts == nullptr) return true;
    if (misaligned(r->slots) || misaligned(r->position) || misaligned(r->offsets) || misaligned(r->counts)) return true;
    return r->rows > 0 && (r->slots == nullptr || r->position == nullptr);
}

int convert(bool to_f8, int dtype, int transpose, int rows, int cols, void *X, int ldx, const int32_t *index,
            const regtile_f8_matrix *Q, void *stream) {
    F8Convert p;
    p.dtype = dtype;
    p.type = Q->type;
    p.block_rows = Q->block_rows;
    p.rows = rows;
    p.cols = cols;
    p.q_rows = Q->rows;
    p.q_cols = Q->cols;
    p.transpose = transpose != 0;
    p.X = X;
    p.ldx = ldx;
    p.index = index;
    p.Q = const_cast<uint8_t *>(Q->codes);
    p.ldq = Q->ld;
    p.S = const_cast<float *>(Q->scales);
    p.s_row = Q->scale_row;
    p.s_col = Q->scale_col;
    if (p.q_rows == 0 || p.q_cols == 0) return regtile::quick();
    (void)hipGetLastError();
    const char *name = "none";
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = to_f8 ? regtile::launch_f8_quantize(p, s, &name) : regtile::launch_f8_dequantize(p, s, &name);
    return regtile::finish(e, name);
}

int run(const F8Problem &p, void *stream) {
    if (p.M == 0 || p.N == 0 || p.experts == 0) return regtile::quick();
    (void)hipGetLastError();
    const char *name = "none";
    const hipError_t e = regtile::launch_f8(p, reinterpret_cast<hipStream_t>(stream), &name);
    return regtile::finish(e, name);
}

// The dense product's problem without C, beta and the workspace; false where the operands do not fit
bool dense(int ta, int tb, const regtile_f8_matrix *A, const regtile_f8_matrix *B, F8Problem *p) {
    *p = F8Problem{};
    p->mode = F8Problem::DENSE;
    p->M = ta ? A->cols : A->rows;
    p->K = ta ? A->rows : A->cols;
    p->N = tb ? B->rows : B->cols;
    p->a = operand(A, ta != 0);
    p->b = operand(B, tb == 0);
    p->experts = 1;
    return (tb ? B->cols : B->rows) == p->K;
}

// ... with its rows, or its depth, in groups
void in_rows(const regtile_expert_rows *rows, int gather, const regtile_f8_matrix *A, const regtile_f8_matrix *B, F8Problem *p) {
    p->mode = F8Problem::ROWS;
    p->M = rows->rows;
    p->experts = rows->experts;
    p->b_stack = B->codes_stack;
    p->bs_stack = B->scales_stack;
    p->offsets = rows->offsets;
    p->counts = rows->counts;
    p->slots = gather ? rows->slots : nullptr;
    p->top_k = rows->k;
    p->a_rows = A->rows;
    p->n_slots = rows->tokens * rows->k;
    p->mean_rows = (int)(((int64_t)p->n_slots + rows->experts - 1) / rows->experts);
}
void in_depth(const regtile_expert_rows *rows, F8Problem *p) {
    p->mode = F8Problem::DEPTH;
    p->experts = rows->experts;
    p->offsets = rows->offsets;
    p->counts = rows->counts;
}

}  // namespace

extern "C" {

int regtile_quantize_f8(int dtype, int transpose, int rows, int cols, const void *X, int ldx, const int32_t *index,
                        const regtile_f8_matrix *Q, void *stream) {
    if (bad_dtype(dtype)) return -1;
    if (transpose != 0 && transpose != 1) return -2;
    if (rows < 0) return -3;
    if (cols < 0) return -4;
    const bool some = Q != nullptr && Q->rows > 0 && Q->cols > 0;
    if ((some && rows > 0 && X == nullptr) || misaligned(X, dtype)) return -5;
    if (ldx < (cols > 1 ? cols : 1)) return -6;
    if (misaligned(index)) return -7;
    if (bad_matrix(Q, true, 1) || (transpose && Q->block_rows != 1)) return -8;
    if ((transpose ? Q->rows : Q->cols) != cols || (index == nullptr && (transpose ? Q->cols : Q->rows) != rows)) return -8;
    return convert(true, dtype, transpose, rows, cols, const_cast<void *>(X), ldx, index, Q, stream);
}

int regtile_dequantize_f8(const regtile_f8_matrix *Q, int dtype, void *X, int ldx, void *stream) {
    if (bad_matrix(Q, true, 1)) return -1;
    if (bad_dtype(dtype)) return -2;
    if ((Q->rows > 0 && Q->cols > 0 && X == nullptr) || misaligned(X, dtype)) return -3;
    if (ldx < (Q->cols > 1 ? Q->cols : 1)) return -4;
    return convert(false, dtype, 0, Q->rows, Q->cols, X, ldx, nullptr, Q, stream);
}

int regtile_gemm_f8(int trans_a, int trans_b, float alpha, const regtile_f8_matrix *A, const regtile_f8_matrix *B, float beta,
                    int c_dtype, void *C, int ldc, void *work, int64_t work_bytes, void *stream) {
    if (trans_a != 0 && trans_a != 1) return -1;
    if (trans_b != 0 && trans_b != 1) return -2;
    if (bad_matrix(A, alpha != 0.0f, 1) || (trans_a && A->block_rows == 1)) return -4;
    if (bad_matrix(B, alpha != 0.0f, 1) || (!trans_b && B->block_rows == 1)) return -5;
    F8Problem p;
    if (!dense(trans_a, trans_b, A, B, &p)) return -5;
    if (bad_dtype(c_dtype)) return -7;
    if ((p.M > 0 && p.N > 0 && C == nullptr) || misaligned(C, c_dtype)) return -8;
    if (ldc < (p.N > 1 ? p.N : 1)) return -9;
    if ((reinterpret_cast<uintptr_t>(work) & 15u) != 0) return -10;
    if (work_bytes < 0 || (work == nullptr && work_bytes != 0)) return -11;
    if (alpha == 0.0f) p.K = 0;
    p.alpha = alpha;
    p.beta = beta;
    p.out.C = C;
    p.out.ldc = ldc;
    p.out.dtype = c_dtype;
    p.work = work;
    p.work_bytes = work_bytes;
    return run(p, stream);
}

int64_t regtile_gemm_f8_workspace(int trans_a, int trans_b, const regtile_f8_matrix *A, const regtile_f8_matrix *B, int c_dtype,
                                  int ldc) {
    F8Problem p;
    if (bad_matrix(A, false, 1) || bad_matrix(B, false, 1) || !dense(trans_a != 0, trans_b != 0, A, B, &p)) return 0;
    if (p.M == 0 || p.N == 0) return 0;
    p.out.ldc = ldc;
    p.out.dtype = c_dtype;
    return regtile::f8_work_bytes(p);
}

int64_t regtile_expert_rows_size(int tokens, int k, int experts, int align) {
    if (tokens < 0 || k < 1 || experts < 1 || align < 1) return -1;
    const int64_t n = (int64_t)tokens * k, most = n < experts ? n : experts;
    const int64_t rows = (n + most * (align - 1) + align - 1) / align * align;
    return n > INT_LIMIT || rows > INT_LIMIT ? -1 : rows;
}

int64_t regtile_order_experts_workspace(int tokens, int k, int experts) {
    return tokens < 0 || k < 1 || experts < 1 ? 0 : regtile::order_work_bytes((int64_t)tokens * k, experts);
}

int regtile_order_experts(const int32_t *chosen, const regtile_expert_rows *rows, void *work, int64_t work_bytes, void *stream) {
    if (bad_rows(rows) || rows->experts > 1024) return -2;
    const int64_t n = (int64_t)rows->tokens * rows->k;
    if ((n > 0 && chosen == nullptr) || misaligned(chosen)) return -1;
    if ((reinterpret_cast<uintptr_t>(work) & 15u) != 0) return -3;
    if (work_bytes < regtile::order_work_bytes(n, rows->experts) || (work == nullptr && work_bytes != 0)) return -4;
    regtile::OrderProblem p;
    p.chosen = chosen;
    p.tokens = rows->tokens;
    p.k = rows->k;
    p.experts = rows->experts;
    p.align = rows->align;
    p.rows = rows->rows;
    p.slots = const_cast<int32_t *>(rows->slots);
    p.position = const_cast<int32_t *>(rows->position);
    p.offsets = const_cast<int32_t *>(rows->offsets);
    p.counts = const_cast<int32_t *>(rows->counts);
    p.work = static_cast<int32_t *>(work);
    (void)hipGetLastError();
    const char *name = "none";
    const hipError_t e = regtile::launch_order(p, reinterpret_cast<hipStream_t>(stream), &name);
    return regtile::finish(e, name);
}

int regtile_gemm_f8_experts(const regtile_expert_rows *rows, int gather, int trans_b, float alpha, const regtile_f8_matrix *A,
                            const regtile_f8_matrix *B, float beta, int c_dtype, void *C, int ldc, void *work, int64_t work_bytes,
                            void *stream) {
    if (bad_rows(rows)) return -1;
    if (gather != 0 && gather != 1) return -2;
    if (trans_b != 0 && trans_b != 1) return -3;
    if (bad_matrix(A, alpha != 0.0f, 1) || A->rows != (gather ? rows->tokens : rows->rows)) return -5;
    if (bad_matrix(B, alpha != 0.0f, rows->experts) || (!trans_b && B->block_rows == 1)) return -6;
    F8Problem p;
    if (!dense(0, trans_b, A, B, &p)) return -6;
    if (bad_dtype(c_dtype)) return -8;
    if ((rows->rows > 0 && p.N > 0 && C == nullptr) || misaligned(C, c_dtype)) return -9;
    if (ldc < (p.N > 1 ? p.N : 1)) return -10;
    if ((reinterpret_cast<uintptr_t>(work) & 15u) != 0) return -11;
    if (work_bytes < 0 || (work == nullptr && work_bytes != 0)) return -12;
    in_rows(rows, gather, A, B, &p);
    if (alpha == 0.0f) p.K = 0;
    p.alpha = alpha;
    p.beta = beta;
    p.out.C = C;
    p.out.ldc = ldc;
    p.out.dtype = c_dtype;
    p.work = work;
    p.work_bytes = work_bytes;
    return run(p, stream);
}

int regtile_gemm_f8_experts_dw(const regtile_expert_rows *rows, float alpha, const regtile_f8_matrix *A, const regtile_f8_matrix *B,
                               float beta, int c_dtype, void *C, int ldc, int64_t c_stack, void *work, int64_t work_bytes,
                               void *stream) {
    if (bad_rows(rows) || rows->align % regtile::f8::BLOCK != 0) return -1;
    if (bad_matrix(A, alpha != 0.0f, 1) || A->cols != rows->rows || A->block_rows != 1) return -3;
    if (bad_matrix(B, alpha != 0.0f, 1) || B->cols != rows->rows || B->block_rows != 1) return -4;
    F8Problem p;
    dense(0, 1, A, B, &p);
    if (bad_dtype(c_dtype)) return -6;
    if ((p.M > 0 && p.N > 0 && C == nullptr) || misaligned(C, c_dtype)) return -7;
    if (ldc < (p.N > 1 ? p.N : 1)) return -8;
    if (c_stack < 0 || (rows->experts > 1 && p.M > 0 && p.N > 0 && c_stack < (int64_t)(p.M - 1) * ldc + p.N)) return -9;
    if ((reinterpret_cast<uintptr_t>(work) & 15u) != 0) return -10;
    if (work_bytes < 0 || (work == nullptr && work_bytes != 0)) return -11;
    in_depth(rows, &p);
    if (alpha == 0.0f) p.K = 0;
    p.alpha = alpha;
    p.beta = beta;
    p.out.C = C;
    p.out.ldc = ldc;
    p.out.dtype = c_dtype;
    p.c_stack = c_stack;
    p.work = work;
    p.work_bytes = work_bytes;
    return run(p, stream);
}

int64_t regtile_gemm_f8_experts_workspace(const regtile_expert_rows *rows, int gather, int trans_b, const regtile_f8_matrix *A,
                                          const regtile_f8_matrix *B, int c_dtype) {
    F8Problem p;
    if (bad_rows(rows) || bad_matrix(A, false, 1) || bad_matrix(B, false, rows->experts) || !dense(0, trans_b != 0, A, B, &p)) return 0;
    if (rows->rows == 0 || p.N == 0 || A->rows != (gather ? rows->tokens : rows->rows)) return 0;
    in_rows(rows, gather, A, B, &p);
    p.out.dtype = c_dtype;
    return regtile::f8_work_bytes(p);
}

int64_t regtile_gemm_f8_experts_dw_workspace(const regtile_expert_rows *rows, const regtile_f8_matrix *A, const regtile_f8_matrix *B,
                                             int c_dtype) {
    F8Problem p;
    if (bad_rows(rows) || bad_matrix(A, false, 1) || bad_matrix(B, false, 1) || !dense(0, 1, A, B, &p)) return 0;
    if (p.M == 0 || p.N == 0 || p.K != rows->rows) return 0;
    in_depth(rows, &p);
    p.out.dtype = c_dtype;
    return regtile::f8_work_bytes(p);
}

int regtile_route_experts(int score, int dtype, int tokens, int experts, int k, int groups, int top_groups, int group_best,
                          int renormalize, float scale, const void *logits, int ldl, const float *bias, int32_t *chosen,
                          float *weights, void *stream) {
    if (score != REGTILE_SCORE_SOFTMAX && score != REGTILE_SCORE_SIGMOID) return -1;
    if (bad_dtype(dtype)) return -2;
    if (tokens < 0) return -3;
    if (experts < 1 || experts > 1024) return -4;
    if (k < 1 || k > 64 || k > experts) return -5;
    if (groups < 1 || groups > 64 || experts % groups != 0) return -6;
    if (top_groups < 1 || top_groups > groups) return -7;
    if (group_best != 1 && group_best != 2) return -8;
    if (renormalize != 0 && renormalize != 1) return -9;
    if ((tokens > 0 && logits == nullptr) || misaligned(logits, dtype)) return -11;
    if (ldl < experts) return -12;
    if (misaligned(bias)) return -13;
    if ((tokens > 0 && chosen == nullptr) || misaligned(chosen)) return -14;
    if ((tokens > 0 && weights == nullptr) || misaligned(weights)) return -15;
    if (tokens == 0) return regtile::quick();
    regtile::RouteProblem p = {};
    p.tokens = tokens;
    p.experts = experts;
    p.k = k;
    p.groups = groups;
    p.top_groups = top_groups;
    p.group_best = group_best;
    p.dtype = dtype;
    p.sigmoid = score == REGTILE_SCORE_SIGMOID;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    p.logits = logits;
    p.ldl = ldl;
    p.bias = bias;
    p.chosen = chosen;
    p.weights = weights;
    (void)hipGetLastError();
    const char *name = "none";
    const hipError_t e = regtile::launch_route(p, reinterpret_cast<hipStream_t>(stream), &name);
    return regtile::finish(e, name);
}

int regtile_route_experts_grad(int score, int dtype, int tokens, int experts, int k, int renormalize, float scale,
                               const void *logits, int ldl, const int32_t *chosen, const float *dweights, void *dlogits, int ldd,
                               void *stream) {
    if (score != REGTILE_SCORE_SOFTMAX && score != REGTILE_SCORE_SIGMOID) return -1;
    if (bad_dtype(dtype)) return -2;
    if (tokens < 0) return -3;
    if (experts < 1 || experts > 1024) return -4;
    if (k < 1 || k > 64 || k > experts) return -5;
    if (renormalize != 0 && renormalize != 1) return -6;
    if ((tokens > 0 && logits == nullptr) || misaligned(logits, dtype)) return -8;
    if (ldl < experts) return -9;
    if ((tokens > 0 && chosen == nullptr) || misaligned(chosen)) return -10;
    if ((tokens > 0 && dweights == nullptr) || misaligned(dweights)) return -11;
    if ((tokens > 0 && dlogits == nullptr) || misaligned(dlogits, dtype)) return -12;
    if (ldd < experts) return -13;
    if (tokens == 0) return regtile::quick();
    regtile::RouteProblem p = {};
    p.tokens = tokens;
    p.experts = experts;
    p.k = k;
    p.dtype = dtype;
    p.sigmoid = score == REGTILE_SCORE_SIGMOID;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    p.logits = logits;
    p.ldl = ldl;
    p.chosen = const_cast<int32_t *>(chosen);
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.ldd = ldd;
    (void)hipGetLastError();
    const char *name = "none";
    const hipError_t e = regtile::launch_route_grad(p, reinterpret_cast<hipStream_t>(stream), &name);
    return regtile::finish(e, name);
}

int regtile_combine_experts(const regtile_expert_rows *rows, int dtype, int n, const void *Y, int ldy, const float *weights, void *out,
                            int ldo, void *stream) {
    if (bad_rows(rows)) return -1;
    if (bad_dtype(dtype)) return -2;
    if (n < 0) return -3;
    const bool some = n > 0 && rows->tokens > 0;
    if ((some && Y == nullptr) || misaligned(Y, dtype)) return -4;
    if (ldy < (n > 1 ? n : 1)) return -5;
    if (misaligned(weights)) return -6;
    if ((some && out == nullptr) || misaligned(out, dtype)) return -7;
    if (ldo < (n > 1 ? n : 1)) return -8;
    if (!some) return regtile::quick();
    regtile::CombineProblem p = {};
    p.tokens = rows->tokens;
    p.k = rows->k;
    p.rows = rows->rows;
    p.n = n;
    p.dtype = dtype;
    p.position = rows->position;
    p.Y = Y;
    p.ldy = ldy;
    p.weights = weights;
    p.out = out;
    p.ldo = ldo;
    (void)hipGetLastError();
    const char *name = "none";
    const hipError_t e = regtile::launch_combine(p, reinterpret_cast<hipStream_t>(stream), &name);
    return regtile::finish(e, name);
}

int regtile_combine_experts_grad(const regtile_expert_rows *rows, int dtype, int n, const void *dout, int ldd, const void *Y, int ldy,
                                 const float *weights, void *dY, int lddy, float *dweights, void *stream) {
    if (bad_rows(rows)) return -1;
    if (bad_dtype(dtype)) return -2;
    if (n < 0) return -3;
    const bool some = n > 0 && rows->rows > 0;
    if ((some && dout == nullptr) || misaligned(dout, dtype)) return -4;
    if (ldd < (n > 1 ? n : 1)) return -5;
    if ((some && dweights != nullptr && Y == nullptr) || misaligned(Y, dtype)) return -6;
    if (dweights != nullptr && ldy < (n > 1 ? n : 1)) return -7;
    if (misaligned(weights)) return -8;
    if ((some && dY == nullptr) || misaligned(dY, dtype)) return -9;
    if (lddy < (n > 1 ? n : 1)) return -10;
    if (misaligned(dweights)) return -11;
    if (rows->rows == 0 || (n == 0 && dweights == nullptr)) return regtile::quick();
    regtile::CombineProblem p = {};
    p.tokens = rows->tokens;
    p.k = rows->k;
    p.rows = rows->rows;
    p.n = n;
    p.dtype = dtype;
    p.slots = rows->slots;
    p.position = rows->position;
    p.Y = Y;
    p.ldy = ldy;
    p.weights = weights;
    p.dout = dout;
    p.ldd = ldd;
    p.dY = dY;
    p.lddy = lddy;
    p.dweights = dweights;
    (void)hipGetLastError();
    const char *name = "none";
    const hipError_t e = regtile::launch_combine_grad(p, reinterpret_cast<hipStream_t>(stream), &name);
    return regtile::finish(e, name);
}

}  // extern "C"
