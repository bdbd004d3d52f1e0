// C ABI entry points: argument validation (host only, before any HIP call),
// variant dispatch and launch-status reporting.  The interface contract is
// documented in include/sgemm.h.
#include <algorithm>
#include <cmath>

#include "../../include/sgemm.h"
#include "kernels.h"

using sgemm::GemmArgs;

namespace {

thread_local int g_last_hip_error = 0;

int launch_status(hipError_t e) {
    if (e == hipSuccess) return SGEMM_OK;
    g_last_hip_error = int(e);
    return SGEMM_ERR_LAUNCH;
}

// Byte range [lo, hi) spanned by a rows x cols row-major view (rows, cols > 0).
void span(const void* p, int64_t rows, int64_t cols, int64_t ld, uintptr_t* lo, uintptr_t* hi) {
    *lo = reinterpret_cast<uintptr_t>(p);
    *hi = *lo + uintptr_t(((rows - 1) * ld + cols) * int64_t(sizeof(float)));
}

bool overlaps(uintptr_t alo, uintptr_t ahi, uintptr_t blo, uintptr_t bhi) {
    return alo < bhi && blo < ahi;
}

int validate(int variant, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
             const float* B, int64_t ldb, const float* C, int64_t ldc) {
    if (variant < 0 || variant >= SGEMM_VARIANT_COUNT) return SGEMM_ERR_VARIANT;
    if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_DIM;
    // Keep every element offset, and (rows - 1) * ld + cols, inside int64.
    const int64_t lim = int64_t(1) << 40;
    if (M > lim || N > lim || K > lim) return SGEMM_ERR_DIM;
    const int64_t k1 = K > 1 ? K : 1, n1 = N > 1 ? N : 1;
    if (lda < k1 || ldb < n1 || ldc < n1) return SGEMM_ERR_LD;
    if (lda > lim || ldb > lim || ldc > lim) return SGEMM_ERR_LD;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr) return SGEMM_ERR_NULLPTR;
    if (K > 0) {
        if (A == nullptr || B == nullptr) return SGEMM_ERR_NULLPTR;
        uintptr_t clo, chi, alo, ahi, blo, bhi;
        span(C, M, N, ldc, &clo, &chi);
        span(A, M, K, lda, &alo, &ahi);
        span(B, K, N, ldb, &blo, &bhi);
        if (overlaps(clo, chi, alo, ahi) || overlaps(clo, chi, blo, bhi)) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

// Validation of the general entry point (row-major; see include/sgemm.h):
// flags, sizes and leading dimensions, then pointers.
int validate_ex_shape(int ta, int tb, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                      int64_t ldc) {
    if ((ta != SGEMM_OP_N && ta != SGEMM_OP_T) || (tb != SGEMM_OP_N && tb != SGEMM_OP_T))
        return SGEMM_ERR_ARG;
    if (M < 0 || N < 0 || K < 0) return SGEMM_ERR_DIM;
    const int64_t lim = int64_t(1) << 40;
    if (M > lim || N > lim || K > lim) return SGEMM_ERR_DIM;
    const int64_t m1 = M > 1 ? M : 1, n1 = N > 1 ? N : 1, k1 = K > 1 ? K : 1;
    if (lda < (ta ? m1 : k1) || ldb < (tb ? k1 : n1) || ldc < n1) return SGEMM_ERR_LD;
    if (lda > lim || ldb > lim || ldc > lim) return SGEMM_ERR_LD;
    return SGEMM_OK;
}

int validate_ex(int ta, int tb, int64_t M, int64_t N, int64_t K, float alpha, const float* A,
                int64_t lda, const float* B, int64_t ldb, const float* C, int64_t ldc) {
    const int v = validate_ex_shape(ta, tb, M, N, K, lda, ldb, ldc);
    if (v != SGEMM_OK) return v;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (C == nullptr) return SGEMM_ERR_NULLPTR;
    if (K > 0 && alpha != 0.0f) {
        if (A == nullptr || B == nullptr) return SGEMM_ERR_NULLPTR;
        uintptr_t clo, chi, alo, ahi, blo, bhi;
        span(C, M, N, ldc, &clo, &chi);
        if (ta) span(A, K, M, lda, &alo, &ahi); else span(A, M, K, lda, &alo, &ahi);
        if (tb) span(B, N, K, ldb, &blo, &bhi); else span(B, K, N, ldb, &blo, &bhi);
        if (overlaps(clo, chi, alo, ahi) || overlaps(clo, chi, blo, bhi)) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

int choose_auto(const GemmArgs& g) {
    // The matrix-core kernel handles every shape whose per-slab offsets fit
    // its 32-bit buffer addressing; the register-tiled kernel (64-bit
    // offsets) takes the rest.
    return sgemm::k4_supports(g) ? SGEMM_K4_MFMA : SGEMM_K3_REGTILE_DB;
}

// A rows x cols row-major view of elements of `size` bytes.
struct View {
    const void* p;
    int64_t rows, cols, ld, size;
};

// Whether two views share an element.  Views of one leading dimension whose
// byte ranges cross may still be disjoint column ranges of one buffer.
bool share(const View& a, const View& b) {
    if (a.rows == 0 || a.cols == 0 || b.rows == 0 || b.cols == 0 || !a.p || !b.p) return false;
    // 128-bit extents: rows * ld may pass 64 bits at the limits above.
    typedef unsigned __int128 wide;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const wide ahi = a0 + (wide(a.rows - 1) * wide(a.ld) + wide(a.cols)) * wide(a.size);
    const wide bhi = b0 + (wide(b.rows - 1) * wide(b.ld) + wide(b.cols)) * wide(b.size);
    if (!(a0 < bhi && b0 < ahi)) return false;
    const int64_t pitch = a.ld * a.size;
    if (pitch != b.ld * b.size) return true;
    // Where b's columns start in a's row pitch: disjoint if they lie wholly
    // in the gap after a's columns.
    const int64_t diff = int64_t(b0 - a0), r = ((diff % pitch) + pitch) % pitch;
    return r < a.cols * a.size || r + b.cols * b.size > pitch;
}

bool same_view(const View& a, const View& b) { return a.p == b.p && a.ld == b.ld; }

// No output shares an element with an input or with another output, except
// that each of the first n_place_out outputs may be exactly one of the first
// n_place inputs.
template <int NI, int NO>
int check_alias(const View (&in)[NI], const View (&out)[NO], int n_place = 0, int n_place_out = 0) {
    for (int o = 0; o < NO; o++) {
        for (int i = 0; i < NI; i++) {
            if (o < n_place_out && i < n_place && same_view(out[o], in[i])) continue;
            if (share(out[o], in[i])) return SGEMM_ERR_ALIAS;
        }
        for (int o2 = 0; o2 < o; o2++)
            if (share(out[o], out[o2])) return SGEMM_ERR_ALIAS;
    }
    return SGEMM_OK;
}

// Whether the last input, a workspace, shares memory with another: kernels write it
// while those are still to be read.
template <int NI>
bool workspace_shared(const View (&in)[NI]) {
    for (int i = 0; i + 1 < NI; i++)
        if (share(in[i], in[NI - 1])) return true;
    return false;
}

constexpr int64_t kDimLimit = int64_t(1) << 40;

bool dims_ok(int64_t a, int64_t b, int64_t c) {
    return a >= 0 && b >= 0 && c >= 0 && a <= kDimLimit && b <= kDimLimit && c <= kDimLimit;
}

bool ld_ok(int64_t ld, int64_t cols) { return ld >= (cols > 1 ? cols : 1) && ld <= kDimLimit; }

int validate_glu(int act, int transw, int64_t M, int64_t F, int64_t K, int64_t ldx, int64_t ldw) {
    if (act < 0 || act >= SGEMM_ACT_COUNT) return SGEMM_ERR_ARG;
    if (transw != SGEMM_OP_N && transw != SGEMM_OP_T) return SGEMM_ERR_ARG;
    if (!dims_ok(M, F, K)) return SGEMM_ERR_DIM;
    if (!ld_ok(ldx, K) || !ld_ok(ldw, transw ? K : F)) return SGEMM_ERR_LD;
    return SGEMM_OK;
}

// The common body of the 4-bit entry points; act < 0: the plain product.
int run_q4(int act, int xtype, int stype, int64_t M, int64_t N, int64_t K, const void* X,
           int64_t ldx, const uint8_t* const (&W)[2], int64_t ldw, int64_t group,
           const void* const (&S)[2], int64_t lds, const uint8_t* const (&Z)[2], int64_t ldz,
           void* Y, int64_t ldy, void* stream) {
    const int nw = act < 0 ? 1 : 2;
    if (xtype < 0 || xtype > SGEMM_TYPE_BF16 || stype < 0 || stype > SGEMM_TYPE_BF16) return SGEMM_ERR_ARG;
    if (group < 32 || (group & (group - 1)) != 0) return SGEMM_ERR_ARG;
    if (nw == 2 && (Z[0] == nullptr) != (Z[1] == nullptr)) return SGEMM_ERR_ARG;
    if (!dims_ok(M, N, K)) return SGEMM_ERR_DIM;
    const int64_t groups = K / group + (K % group != 0), bytes = (K + 1) / 2;
    if (!ld_ok(ldx, K) || !ld_ok(ldw, bytes) || !ld_ok(lds, groups) || !ld_ok(ldy, N)) return SGEMM_ERR_LD;
    if (Z[0] && !ld_ok(ldz, groups)) return SGEMM_ERR_LD;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (Y == nullptr) return SGEMM_ERR_NULLPTR;
    const int64_t xs = xtype == SGEMM_TYPE_F32 ? 4 : 2, ss = stype == SGEMM_TYPE_F32 ? 4 : 2;
    if (K > 0) {
        if (X == nullptr) return SGEMM_ERR_NULLPTR;
        for (int i = 0; i < nw; i++)
            if (W[i] == nullptr || S[i] == nullptr) return SGEMM_ERR_NULLPTR;
        const View in[] = {{X, M, K, ldx, xs},         {W[0], N, bytes, ldw, 1}, {S[0], N, groups, lds, ss},
                           {Z[0], N, groups, ldz, 1}, {W[1], N, bytes, ldw, 1}, {S[1], N, groups, lds, ss},
                           {Z[1], N, groups, ldz, 1}};
        const View out[] = {{Y, M, N, ldy, xs}};
        const int a = check_alias(in, out);
        if (a != SGEMM_OK) return a;
    }
    sgemm::Q4Args g{};
    g.act = act;
    g.xtype = xtype;
    g.stype = stype;
    g.shift = 0;
    while ((int64_t(1) << g.shift) < group) g.shift++;
    g.M = M;
    g.N = N;
    g.K = K;
    g.X = X;
    g.ldx = ldx;
    g.ldw = ldw;
    g.lds = lds;
    g.ldz = ldz;
    g.Y = Y;
    g.ldy = ldy;
    for (int i = 0; i < 2; i++) {
        g.W[i] = W[i];
        g.S[i] = S[i];
        g.Z[i] = Z[i];
    }
    return launch_status(sgemm::launch_q4(g, static_cast<hipStream_t>(stream)));
}

// A stack of `n` rows x cols matrices, `stride` elements apart; of more than
// one, the one row of elements that they span.
View stack_view(const void* p, int64_t n, int64_t stride, int64_t rows, int64_t cols, int64_t ld,
                int64_t size) {
    if (!p || n <= 0 || rows <= 0 || cols <= 0) return {nullptr, 0, 0, 1, size};
    if (n == 1) return {p, rows, cols, ld, size};
    const int64_t len = (n - 1) * stride + (rows - 1) * ld + cols;
    return {p, 1, len, len, size};
}

// Whether a stack's strides keep every element inside 62 bits of offset (and,
// for an output, its matrices apart).
bool stack_ok(int64_t n, int64_t stride, int64_t rows, int64_t cols, int64_t ld, bool output) {
    if (!ld_ok(ld, cols) || stride < 0 || stride > (int64_t(1) << 60)) return false;
    typedef __int128 wide;
    const wide one = rows > 0 ? wide(rows - 1) * ld + cols : 0;
    if (wide(n > 0 ? n - 1 : 0) * stride + one > (wide(1) << 60)) return false;
    // Apart: one after another, or rows of one matrix in the gaps of another's.
    return !output || n <= 1 || stride >= one ||
           (stride >= cols && (n - 1) * wide(stride) + cols <= ld);
}

constexpr int64_t kIndexLimit = (int64_t(1) << 31) - 1;
constexpr int64_t kOrthoLimit = SGEMM_ORTHO_MAX_SIDE, kOrthoBatch = SGEMM_ORTHO_MAX_BATCH;

int validate_lora_sizes(int type, int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
    if (type < 0 || type > SGEMM_TYPE_BF16) return SGEMM_ERR_ARG;
    if (M < 0 || N < 0 || K < 0 || M > kIndexLimit || N > kIndexLimit || K > kIndexLimit) return SGEMM_ERR_DIM;
    if (R < 1 || R > SGEMM_LORA_MAX_RANK || L < 1 || L > SGEMM_LORA_MAX_ADAPTERS) return SGEMM_ERR_DIM;
    return SGEMM_OK;
}

// Bound of the singular values after each step (bounds[i]: before step i), from
// those of G / |G|, which are at most 1.  |a s + b s^3 + c s^5| over [0, r] is
// largest at r or where a + 3 b q + 5 c q^2 = 0, q = s^2.
bool ortho_bounds(int steps, const double* coef, double* bounds) {
    double r = 1.0;
    for (int i = 0; i < steps; i++) {
        const double a = coef[3 * i], b = coef[3 * i + 1], c = coef[3 * i + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        bounds[i] = r;
        // The factor a + b s^2 + c s^4 is stored too.  (Also no square below overflows.)
        if (!(std::fabs(a) + std::fabs(b) * r * r + std::fabs(c) * std::pow(r, 4) <= 1e9)) return false;
        auto p = [&](double q) { return std::fabs(std::sqrt(q) * (a + q * (b + q * c))); };
        double top = p(r * r);
        const double disc = 9 * b * b - 20 * a * c;
        if (disc >= 0) {
            // No difference of nearly equal numbers: a root far smaller than the other
            // keeps its digits.  Where c or t is zero one is infinite or NaN, and not taken.
            const double t = -(3 * b + std::copysign(std::sqrt(disc), b)) / 2;
            for (double q : {t / (5 * c), a / t})
                if (q > 0 && q < r * r) top = std::max(top, p(q));
        }
        // Roundings of a step and of its result, counted generously.
        r = top * 1.01;
        if (!(r <= 64.0) || r < 0x1p-40) return false;
    }
    bounds[steps] = r;
    return true;
}

}  // namespace

extern "C" {

int sgemm_f32_variant(int variant, int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                      const float* B, int64_t ldb, float* C, int64_t ldc, void* stream) {
    const int v = validate(variant, M, N, K, A, lda, B, ldb, C, ldc);
    if (v != SGEMM_OK) return v;
    if (M == 0 || N == 0) return SGEMM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const GemmArgs g{M, N, K, A, lda, B, ldb, C, ldc};
    if (K == 0) return launch_status(sgemm::launch_zero(C, M, N, ldc, s));
    if (variant == SGEMM_AUTO) {
        // AUTO may also take the thin-product kernels (vector units) for
        // products with one side of C at most 8.
        if (choose_auto(g) == SGEMM_K4_MFMA) return launch_status(sgemm::launch_k4_mfma(g, s, 0, true));
        return launch_status(sgemm::launch_k3_regtile(g, s));
    }
    switch (variant) {
        case SGEMM_K0_NAIVE: return launch_status(sgemm::launch_k0_naive(g, s));
        case SGEMM_K1_COALESCED: return launch_status(sgemm::launch_k1_coalesced(g, s));
        case SGEMM_K2_LDS_TILED: return launch_status(sgemm::launch_k2_lds(g, 32, 0, s));
        case SGEMM_K2_LDS_TILED16: return launch_status(sgemm::launch_k2_lds(g, 16, 0, s));
        case SGEMM_K2_LDS_TILED_PAD1: return launch_status(sgemm::launch_k2_lds(g, 32, 1, s));
        case SGEMM_K2_LDS_TILED16_PAD1: return launch_status(sgemm::launch_k2_lds(g, 16, 1, s));
        case SGEMM_K3_REGTILE_DB: return launch_status(sgemm::launch_k3_regtile(g, s));
        case SGEMM_K4_MFMA:
            if (!sgemm::k4_supports(g)) return SGEMM_ERR_UNSUPPORTED;
            // Always the matrix cores (tile, K split and packing by shape).
            return launch_status(sgemm::launch_k4_mfma(g, s, 0, false));
        case SGEMM_K4_MFMA_TILE128:
            if (!sgemm::k4_supports(g)) return SGEMM_ERR_UNSUPPORTED;
            return launch_status(sgemm::launch_k4_tile128(g, s));
        case SGEMM_K4_MFMA_TILE64:
            if (!sgemm::k4_supports(g)) return SGEMM_ERR_UNSUPPORTED;
            return launch_status(sgemm::launch_k4_tile64(g, s));
        case SGEMM_K4_MFMA_TILE128X256:
            if (!sgemm::k4_supports(g)) return SGEMM_ERR_UNSUPPORTED;
            return launch_status(sgemm::launch_k4_tile128x256(g, s));
        default: return SGEMM_ERR_VARIANT;
    }
}

int sgemm_f32(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda, const float* B,
              int64_t ldb, float* C, int64_t ldc, void* stream) {
    return sgemm_f32_variant(SGEMM_AUTO, M, N, K, A, lda, B, ldb, C, ldc, stream);
}

int sgemm_f32_ex_split(int transa, int transb, int64_t M, int64_t N, int64_t K, float alpha,
                       const float* A, int64_t lda, const float* B, int64_t ldb, float beta,
                       float* C, int64_t ldc, int splits, void* stream) {
    if (splits < 0 || splits > SGEMM_MAX_SPLITS) return SGEMM_ERR_ARG;
    const int v = validate_ex(transa, transb, M, N, K, alpha, A, lda, B, ldb, C, ldc);
    if (v != SGEMM_OK) return v;
    if (M == 0 || N == 0) return SGEMM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0 || alpha == 0.0f) return launch_status(sgemm::launch_scale(C, M, N, ldc, beta, s));
    GemmArgs g{M, N, K, A, lda, B, ldb, C, ldc};
    g.trans_a = transa == SGEMM_OP_T;
    g.trans_b = transb == SGEMM_OP_T;
    g.alpha = alpha;
    g.beta = beta;
    if (sgemm::k4_supports(g)) return launch_status(sgemm::launch_k4_mfma(g, s, splits));
    return launch_status(sgemm::launch_k1_general(g, s));
}

int sgemm_f32_ex_split_noalloc(int transa, int transb, int64_t M, int64_t N, int64_t K,
                               float alpha, const float* A, int64_t lda, const float* B,
                               int64_t ldb, float beta, float* C, int64_t ldc, int splits,
                               void* stream) {
    static_assert(sgemm::kStaticScratchBytes == size_t(SGEMM_STATIC_SCRATCH_BYTES),
                  "header and library agree on the static scratch size");
    if (splits < 0 || splits > SGEMM_MAX_SPLITS) return SGEMM_ERR_ARG;
    const int v = validate_ex(transa, transb, M, N, K, alpha, A, lda, B, ldb, C, ldc);
    if (v != SGEMM_OK) return v;
    if (M == 0 || N == 0) return SGEMM_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0 || alpha == 0.0f) return launch_status(sgemm::launch_scale(C, M, N, ldc, beta, s));
    GemmArgs g{M, N, K, A, lda, B, ldb, C, ldc};
    g.trans_a = transa == SGEMM_OP_T;
    g.trans_b = transb == SGEMM_OP_T;
    g.alpha = alpha;
    g.beta = beta;
    if (!sgemm::k4_supports(g)) return launch_status(sgemm::launch_k1_general(g, s));
    // An explicit split whose partial products exceed the scratch is refused
    // before any HIP call.
    if (splits >= 2 && sgemm::k4_split_scratch_bytes(g, splits) > sgemm::kStaticScratchBytes)
        return SGEMM_ERR_SCRATCH;
    sgemm::FixedScratch fs;
    const hipError_t e = sgemm::static_scratch(s, &fs);
    if (e != hipSuccess) return launch_status(e);
    return launch_status(sgemm::launch_k4_mfma(g, s, splits, true, &fs));
}

int sgemm_f32_ex(int transa, int transb, int64_t M, int64_t N, int64_t K, float alpha,
                 const float* A, int64_t lda, const float* B, int64_t ldb, float beta, float* C,
                 int64_t ldc, void* stream) {
    return sgemm_f32_ex_split(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, 0,
                              stream);
}

int sgemm_f32_colmajor(int transa, int transb, int64_t m, int64_t n, int64_t k, float alpha,
                       const float* A, int64_t lda, const float* B, int64_t ldb, float beta,
                       float* C, int64_t ldc, void* stream) {
    // A column-major m x n matrix read row-major is its transpose, so
    // C = op(A) op(B) (column-major) is C^T = op(B)^T op(A)^T (row-major):
    // the operands swap places and keep their transpose flags.
    return sgemm_f32_ex(transb, transa, n, m, k, alpha, B, ldb, A, lda, beta, C, ldc, stream);
}

int sgemm_glu_f32(int act, int transw, int64_t M, int64_t F, int64_t K, const float* X,
                  int64_t ldx, const float* Wg, const float* Wu, int64_t ldw, float* H, int64_t ldh,
                  float* G, float* U, int64_t ldgu, void* stream) {
    int v = validate_glu(act, transw, M, F, K, ldx, ldw);
    if (v != SGEMM_OK) return v;
    if ((G == nullptr) != (U == nullptr)) return SGEMM_ERR_ARG;
    if (!ld_ok(ldh, F) || (G && !ld_ok(ldgu, F))) return SGEMM_ERR_LD;
    if (M == 0 || F == 0) return SGEMM_OK;
    if (H == nullptr || (K > 0 && (!X || !Wg || !Wu))) return SGEMM_ERR_NULLPTR;
    const int64_t wr = transw ? F : K, wc = transw ? K : F;
    const View in[] = {{X, M, K, ldx, 4}, {Wg, wr, wc, ldw, 4}, {Wu, wr, wc, ldw, 4}};
    const View out[] = {{H, M, F, ldh, 4}, {G, M, F, ldgu, 4}, {U, M, F, ldgu, 4}};
    if ((v = check_alias(in, out)) != SGEMM_OK) return v;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (K == 0) {
        hipError_t e = sgemm::launch_zero(H, M, F, ldh, s);
        if (e == hipSuccess && G) e = sgemm::launch_zero(G, M, F, ldgu, s);
        if (e == hipSuccess && U) e = sgemm::launch_zero(U, M, F, ldgu, s);
        return launch_status(e);
    }
    const sgemm::GluArgs g{act, transw == SGEMM_OP_T, M, F, K, X, ldx, Wg, Wu, ldw, H, ldh, G, U, ldgu};
    return launch_status(sgemm::launch_glu(g, s));
}

int sgemm_glu_backward_f32(int act, int transw, int64_t M, int64_t F, int64_t K, const float* X,
                           int64_t ldx, const float* Wg, const float* Wu, int64_t ldw,
                           const float* G, const float* U, int64_t ldgu, const float* dH,
                           int64_t lddh, float* dG, float* dU, int64_t lddgu, float* dX,
                           int64_t lddx, float* dWg, float* dWu, int64_t lddw, float beta,
                           void* stream) {
    int v = validate_glu(act, transw, M, F, K, ldx, ldw);
    if (v != SGEMM_OK) return v;
    if ((dWg == nullptr) != (dWu == nullptr)) return SGEMM_ERR_ARG;
    const int64_t wr = transw ? F : K, wc = transw ? K : F;
    if (!ld_ok(ldgu, F) || !ld_ok(lddh, F) || !ld_ok(lddgu, F)) return SGEMM_ERR_LD;
    if ((dX && !ld_ok(lddx, K)) || (dWg && !ld_ok(lddw, wc))) return SGEMM_ERR_LD;
    const bool some = M > 0 && F > 0;
    if (some && (!G || !U || !dH || !dG || !dU)) return SGEMM_ERR_NULLPTR;
    if (some && K > 0 && ((dX && (!Wg || !Wu)) || (dWg && !X))) return SGEMM_ERR_NULLPTR;
    const View in[] = {{G, M, F, ldgu, 4}, {U, M, F, ldgu, 4},   {dH, M, F, lddh, 4},
                       {X, M, K, ldx, 4},  {Wg, wr, wc, ldw, 4}, {Wu, wr, wc, ldw, 4}};
    const View out[] = {{dG, M, F, lddgu, 4}, {dU, M, F, lddgu, 4},    {dX, M, K, lddx, 4},
                        {dWg, wr, wc, lddw, 4}, {dWu, wr, wc, lddw, 4}};
    if ((v = check_alias(in, out, 3, 2)) != SGEMM_OK) return v;
    const sgemm::GluGradArgs g{act, transw == SGEMM_OP_T, M,  F,  K,     X,  ldx,  Wg,  Wu,  ldw,  G,    U,
                               ldgu, dH, lddh, dG, dU, lddgu, dX, lddx, dWg, dWu, lddw, beta};
    return launch_status(sgemm::launch_glu_backward(g, static_cast<hipStream_t>(stream)));
}

int sgemm_q4(int xtype, int stype, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
             const uint8_t* Wq, int64_t ldw, int64_t group, const void* S, int64_t lds,
             const uint8_t* Z, int64_t ldz, void* Y, int64_t ldy, void* stream) {
    return run_q4(-1, xtype, stype, M, N, K, X, ldx, {Wq, nullptr}, ldw, group, {S, nullptr}, lds,
                  {Z, nullptr}, ldz, Y, ldy, stream);
}

int sgemm_q4_glu(int act, int xtype, int stype, int64_t M, int64_t F, int64_t K, const void* X,
                 int64_t ldx, const uint8_t* Wg, const uint8_t* Wu, int64_t ldw, int64_t group,
                 const void* Sg, const void* Su, int64_t lds, const uint8_t* Zg, const uint8_t* Zu,
                 int64_t ldz, void* H, int64_t ldh, void* stream) {
    if (act < 0 || act >= SGEMM_ACT_COUNT) return SGEMM_ERR_ARG;
    return run_q4(act, xtype, stype, M, F, K, X, ldx, {Wg, Wu}, ldw, group, {Sg, Su}, lds, {Zg, Zu},
                  ldz, H, ldh, stream);
}

int64_t sgemm_lora_workspace(int backward, int type, int64_t M, int64_t N, int64_t K, int64_t R,
                             int64_t L) {
    const int v = validate_lora_sizes(type, M, N, K, R, L);
    if (v != SGEMM_OK) return -v;
    return int64_t(sgemm::lora_workspace_bytes(backward != 0, type, M, N, K, int(R), int(L)));
}

int sgemm_lora(int type, int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, const void* X,
               int64_t ldx, const void* A, int64_t lda, int64_t stride_a, const void* B, int64_t ldb,
               int64_t stride_b, const void* ids, int id_bits, const float* s, float alpha,
               const void* base, int64_t ldbase, void* Y, int64_t ldy, float* H, int64_t ldh,
               void* workspace, int64_t workspace_bytes, void* stream) {
    int v = validate_lora_sizes(type, M, N, K, R, L);
    if (v != SGEMM_OK) return v;
    if (id_bits != 32 && id_bits != 64) return SGEMM_ERR_ARG;
    if (!ld_ok(ldx, K) || !ld_ok(ldy, N) || (base && !ld_ok(ldbase, N)) || (H && !ld_ok(ldh, R))) return SGEMM_ERR_LD;
    if (!stack_ok(L, stride_a, R, K, lda, false) || !stack_ok(L, stride_b, N, R, ldb, false)) return SGEMM_ERR_LD;
    if (M == 0 || (N == 0 && !H)) return SGEMM_OK;
    if ((N > 0 && (!Y || !B)) || (K > 0 && (!X || !A))) return SGEMM_ERR_NULLPTR;
    const int64_t es = type == SGEMM_TYPE_F32 ? 4 : 2;
    const View in[] = {{base, M, N, ldbase, es}, {X, M, K, ldx, es}, stack_view(A, L, stride_a, R, K, lda, es),
                       stack_view(B, L, stride_b, N, R, ldb, es), {ids, 1, M, M, id_bits / 8}, {s, 1, L, L, 4},
                       {workspace, 1, workspace_bytes, workspace_bytes > 0 ? workspace_bytes : 1, 1}};
    const View out[] = {{Y, M, N, ldy, es}, {H, M, R, ldh, 4}};
    if ((v = check_alias(in, out, 1, 1)) != SGEMM_OK) return v;
    if (workspace_shared(in)) return SGEMM_ERR_ALIAS;
    if (workspace_bytes < int64_t(sgemm::lora_workspace_bytes(false, type, M, N, K, int(R), int(L))))
        return SGEMM_ERR_SCRATCH;
    if (workspace_bytes > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15))) return SGEMM_ERR_ARG;
    const sgemm::LoraArgs g{type, M,  N,  K,  int(R), int(L),        X,  ldx,   A,    lda,    stride_a, B,
                            ldb,  stride_b, ids, id_bits == 64, s, alpha, base, ldbase, Y, ldy, H, ldh, workspace};
    return launch_status(sgemm::launch_lora(g, static_cast<hipStream_t>(stream)));
}

int sgemm_lora_backward(int type, int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                        const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* A,
                        int64_t lda, int64_t stride_a, const void* B, int64_t ldb, int64_t stride_b,
                        const float* H, int64_t ldh, const void* ids, int id_bits, const float* s,
                        float alpha, const void* base, int64_t ldbase, void* dX, int64_t lddx,
                        void* dA, int64_t ldda, int64_t stride_da, void* dB, int64_t lddb,
                        int64_t stride_db, void* workspace, int64_t workspace_bytes, void* stream) {
    int v = validate_lora_sizes(type, M, N, K, R, L);
    if (v != SGEMM_OK) return v;
    if (id_bits != 32 && id_bits != 64) return SGEMM_ERR_ARG;
    if (!ld_ok(lddy, N) || !ld_ok(ldx, K) || !ld_ok(ldh, R) || (base && !ld_ok(ldbase, K)) || (dX && !ld_ok(lddx, K)))
        return SGEMM_ERR_LD;
    if (!stack_ok(L, stride_a, R, K, lda, false) || !stack_ok(L, stride_b, N, R, ldb, false)) return SGEMM_ERR_LD;
    if ((dA && !stack_ok(L, stride_da, R, K, ldda, true)) || (dB && !stack_ok(L, stride_db, N, R, lddb, true)))
        return SGEMM_ERR_LD;
    if (!dX && !dA && !dB) return SGEMM_OK;
    const bool rows = M > 0;
    if (rows && N > 0 && (!dY || ((dX || dA) && !B) || (dB && !H))) return SGEMM_ERR_NULLPTR;
    if (rows && K > 0 && ((dX && !A) || (dA && !X))) return SGEMM_ERR_NULLPTR;
    const int64_t es = type == SGEMM_TYPE_F32 ? 4 : 2;
    const View in[] = {{base, M, K, ldbase, es}, {X, M, K, ldx, es}, {dY, M, N, lddy, es},
                       stack_view(A, L, stride_a, R, K, lda, es), stack_view(B, L, stride_b, N, R, ldb, es),
                       {H, M, R, ldh, 4}, {ids, 1, M, M > 0 ? M : 1, id_bits / 8}, {s, 1, L, L, 4},
                       {workspace, 1, workspace_bytes, workspace_bytes > 0 ? workspace_bytes : 1, 1}};
    const View out[] = {{dX, M, K, lddx, es}, stack_view(dA, L, stride_da, R, K, ldda, es),
                        stack_view(dB, L, stride_db, N, R, lddb, es)};
    if ((v = check_alias(in, out, 1, 1)) != SGEMM_OK) return v;
    if (workspace_shared(in)) return SGEMM_ERR_ALIAS;
    if (workspace_bytes < int64_t(sgemm::lora_workspace_bytes(true, type, M, N, K, int(R), int(L))))
        return SGEMM_ERR_SCRATCH;
    if (workspace_bytes > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15))) return SGEMM_ERR_ARG;
    const sgemm::LoraGradArgs g{{type, M, N, K, int(R), int(L), X, ldx, A, lda, stride_a, B, ldb, stride_b, ids,
                                 id_bits == 64, s, alpha, base, ldbase, const_cast<void*>(dY), lddy,
                                 const_cast<float*>(H), ldh, workspace},
                                dX, lddx, dA, ldda, stride_da, dB, lddb, stride_db};
    return launch_status(sgemm::launch_lora_backward(g, static_cast<hipStream_t>(stream)));
}

int64_t sgemm_orthogonalize_workspace(int64_t batch, int64_t M, int64_t N) {
    if (batch < 0 || M < 0 || N < 0 || M > kOrthoLimit || N > kOrthoLimit || batch > kOrthoBatch) return -SGEMM_ERR_DIM;
    return int64_t(sgemm::ortho_workspace_bytes(batch, M, N));
}

int sgemm_orthogonalize(int type, int64_t batch, int64_t M, int64_t N, const void* G, int64_t ldg,
                        int64_t stride_g, void* O, int64_t ldo, int64_t stride_o, int steps,
                        const double* coefficients, double eps, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    if (type < 0 || type > SGEMM_TYPE_BF16 || steps < 1 || steps > SGEMM_ORTHO_MAX_STEPS) return SGEMM_ERR_ARG;
    if (!(eps >= 0) || !std::isfinite(eps)) return SGEMM_ERR_ARG;
    if (batch < 0 || M < 0 || N < 0 || M > kOrthoLimit || N > kOrthoLimit || batch > kOrthoBatch) return SGEMM_ERR_DIM;
    if (!stack_ok(batch, stride_g, M, N, ldg, false) || !stack_ok(batch, stride_o, M, N, ldo, true)) return SGEMM_ERR_LD;
    if (!coefficients) return SGEMM_ERR_NULLPTR;
    double bounds[SGEMM_ORTHO_MAX_STEPS + 1];
    if (!ortho_bounds(steps, coefficients, bounds)) return SGEMM_ERR_ARG;
    if (batch == 0 || M == 0 || N == 0) return SGEMM_OK;
    if (!G || !O) return SGEMM_ERR_NULLPTR;
    const int64_t es = type == SGEMM_TYPE_F32 ? 4 : 2;
    const bool place = G == O && ldg == ldo && (batch == 1 || stride_g == stride_o);
    const View w{workspace, 1, workspace_bytes, workspace_bytes > 0 ? workspace_bytes : 1, 1};
    const View vg = stack_view(G, batch, stride_g, M, N, ldg, es), vo = stack_view(O, batch, stride_o, M, N, ldo, es);
    if ((!place && share(vg, vo)) || share(vg, w) || share(vo, w)) return SGEMM_ERR_ALIAS;
    if (workspace_bytes < int64_t(sgemm::ortho_workspace_bytes(batch, M, N))) return SGEMM_ERR_SCRATCH;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return SGEMM_ERR_ARG;
    const sgemm::OrthoArgs g{type, batch, M,     N,   G,      ldg, stride_g, O,
                             ldo,  stride_o, steps, coefficients, bounds, eps, workspace};
    return launch_status(sgemm::launch_orthogonalize(g, static_cast<hipStream_t>(stream)));
}

int sgemm_auto_variant(int64_t M, int64_t N, int64_t K, const float* A, int64_t lda,
                       const float* B, int64_t ldb, float* C, int64_t ldc) {
    const int v = validate(SGEMM_AUTO, M, N, K, A, lda, B, ldb, C, ldc);
    if (v != SGEMM_OK) return -v;
    const GemmArgs g{M, N, K, A, lda, B, ldb, C, ldc};
    return choose_auto(g);
}

int sgemm_split_plan(int transa, int transb, int64_t M, int64_t N, int64_t K, const float* A,
                     int64_t lda, const float* B, int64_t ldb, int splits, int64_t* kchunk) {
    if (splits < 0 || splits > SGEMM_MAX_SPLITS) return -SGEMM_ERR_ARG;
    const int v = validate_ex_shape(transa, transb, M, N, K, lda, ldb, N > 1 ? N : 1);
    if (v != SGEMM_OK) return -v;
    GemmArgs g{M, N, K, A, lda, B, ldb, nullptr, N > 1 ? N : 1};
    g.trans_a = transa == SGEMM_OP_T;
    g.trans_b = transb == SGEMM_OP_T;
    sgemm::PlanInfo p;
    p.splits = 1;
    p.kchunk = K;
    if (M > 0 && N > 0 && K > 0 && sgemm::k4_supports(g)) p = sgemm::plan_info(g, splits);
    if (kchunk) *kchunk = p.kchunk;
    return p.splits;
}

int sgemm_plan_config(int transa, int transb, int64_t M, int64_t N, int64_t K, const float* A,
                      int64_t lda, const float* B, int64_t ldb, int* engine, int* tile_m,
                      int* tile_n, int* k_groups, int* packed, int64_t* kchunk) {
    const int v = validate_ex_shape(transa, transb, M, N, K, lda, ldb, N > 1 ? N : 1);
    if (v != SGEMM_OK) return -v;
    GemmArgs g{M, N, K, A, lda, B, ldb, nullptr, N > 1 ? N : 1};
    g.trans_a = transa == SGEMM_OP_T;
    g.trans_b = transb == SGEMM_OP_T;
    sgemm::PlanInfo p;
    if (M > 0 && N > 0 && K > 0 && sgemm::k4_supports(g)) p = sgemm::plan_info(g, 0);
    if (engine) *engine = p.engine;
    if (tile_m) *tile_m = p.tile_m;
    if (tile_n) *tile_n = p.tile_n;
    if (k_groups) *k_groups = p.k_groups;
    if (packed) *packed = p.packed ? 1 : 0;
    if (kchunk) *kchunk = p.kchunk;
    return p.splits;
}

int sgemm_copy_f32_launch(float* dst, const float* src, int64_t n, int block, int64_t grid,
                          void* stream) {
    if (n < 0) return SGEMM_ERR_ARG;
    if (block < 64 || block > 1024 || block % 64 != 0) return SGEMM_ERR_ARG;
    if (grid < 1 || grid > sgemm::kMaxCopyGrid) return SGEMM_ERR_ARG;
    if (n == 0) return SGEMM_OK;
    if (dst == nullptr || src == nullptr) return SGEMM_ERR_NULLPTR;
    const uintptr_t d = reinterpret_cast<uintptr_t>(dst), s = reinterpret_cast<uintptr_t>(src);
    const uintptr_t bytes = uintptr_t(n) * sizeof(float);
    if (overlaps(d, d + bytes, s, s + bytes)) return SGEMM_ERR_ALIAS;
    return launch_status(sgemm::launch_copy(dst, src, n, block, grid,
                                            static_cast<hipStream_t>(stream)));
}

int sgemm_copy_f32(float* dst, const float* src, int64_t n, void* stream) {
    const int block = sgemm::kCopyBlock;
    return sgemm_copy_f32_launch(dst, src, n, block, sgemm::copy_default_grid(n, block), stream);
}

int sgemm_probe_valu_f32(float* out, int64_t blocks, int block, int64_t iters, float x, float y,
                         void* stream) {
    if (blocks < 1 || blocks > sgemm::kMaxGrid) return SGEMM_ERR_ARG;
    if (block < 64 || block > 1024 || block % 64 != 0) return SGEMM_ERR_ARG;
    if (iters < 0) return SGEMM_ERR_ARG;
    if (out == nullptr) return SGEMM_ERR_NULLPTR;
    return launch_status(sgemm::launch_probe_valu(out, iters, x, y, blocks, block,
                                                  static_cast<hipStream_t>(stream)));
}

int sgemm_probe_mfma_f32(float* out, const float* a_vals, const float* b_vals, int64_t blocks,
                         int64_t iters, void* stream) {
    if (blocks < 1 || blocks > sgemm::kMaxGrid) return SGEMM_ERR_ARG;
    if (iters < 0) return SGEMM_ERR_ARG;
    if (out == nullptr || a_vals == nullptr || b_vals == nullptr) return SGEMM_ERR_NULLPTR;
    return launch_status(sgemm::launch_probe_mfma(out, a_vals, b_vals, iters, blocks,
                                                  static_cast<hipStream_t>(stream)));
}

const char* sgemm_status_string(int status) {
    switch (status) {
        case SGEMM_OK: return "ok";
        case SGEMM_ERR_DIM: return "invalid dimension (M, N and K must be >= 0)";
        case SGEMM_ERR_LD: return "invalid leading dimension (lda >= max(1,K), ldb and ldc >= max(1,N))";
        case SGEMM_ERR_NULLPTR: return "null operand pointer";
        case SGEMM_ERR_VARIANT: return "unknown kernel variant";
        case SGEMM_ERR_ALIAS: return "output overlaps an input";
        case SGEMM_ERR_LAUNCH: return "kernel launch failed";
        case SGEMM_ERR_UNSUPPORTED: return "variant cannot address this shape";
        case SGEMM_ERR_ARG: return "invalid argument";
        case SGEMM_ERR_SCRATCH: return "scratch memory too small (the static scratch for a requested split, or the workspace given)";
        default: return "unknown status";
    }
}

const char* sgemm_variant_name(int variant) {
    switch (variant) {
        case SGEMM_AUTO: return "auto";
        case SGEMM_K1_COALESCED: return "k1_coalesced";
        case SGEMM_K2_LDS_TILED: return "k2_lds_tiled32";
        case SGEMM_K2_LDS_TILED16_PAD1: return "k2_lds_tiled16_pad1";
        case SGEMM_K3_REGTILE_DB: return "k3_regtile_db";
        case SGEMM_K4_MFMA: return "k4_mfma";
        case SGEMM_K2_LDS_TILED16: return "k2_lds_tiled16";
        case SGEMM_K2_LDS_TILED_PAD1: return "k2_lds_tiled32_pad1";
        case SGEMM_K0_NAIVE: return "k0_naive";
        case SGEMM_K4_MFMA_TILE128: return "k4_mfma_tile128";
        case SGEMM_K4_MFMA_TILE64: return "k4_mfma_tile64";
        case SGEMM_K4_MFMA_TILE128X256: return "k4_mfma_tile128x256";
        default: return nullptr;
    }
}

int sgemm_last_hip_error(void) { return g_last_hip_error; }

int sgemm_abi_version(void) { return SGEMM_ABI_VERSION; }

}  // extern "C"
