// Host check of the gated form's layouts (k4::Cfg with GLU): both weights'
// elements are staged once each where the fragment reads look for them, a
// wave's blocks pair the same columns of both, and the epilogue's pieces cover
// its outputs once.
#include <cstdio>
#include <map>
#include <set>
#include <tuple>
#include <vector>

#include "../roofline_sgemm_f32_amd/csrc/k4_layout.h"

using namespace sgemm::k4;

static int failures = 0;
#define CHECK(c, ...)                                      \
    do {                                                   \
        if (!(c)) {                                        \
            if (failures++ < 20) { printf(__VA_ARGS__); printf("\n"); } \
        }                                                  \
    } while (0)

template <class CF>
void check(const char* name) {
    using LB = typename CF::LB;
    // Staging as the kernel issues it.
    std::map<int, std::tuple<int, int, int>> at;  // byte -> (matrix, column, k)
    for (int wave = 0; wave < CF::NWAVES; wave++)
        for (int q = 0; q < CF::B_INSTR_PER_WAVE; q++) {
            const int uu = wave * CF::B_INSTR_PER_WAVE + q, u = uu % LB::INSTR, image = uu / LB::INSTR;
            CHECK(image < 2, "%s load instruction past both images", name);
            for (int lane = 0; lane < 64; lane++)
                for (int e = 0; e < LB::LSIZE / 4; e++) {
                    const int byte = CF::B_BASE + image * LB::STAGE + LB::load_lds(u) + lane * LB::LSIZE + 4 * e;
                    int col, k;
                    if constexpr (CF::B_KMAJOR) {
                        col = LB::load_row(u, lane);
                        k = LB::load_k(u, lane) + e;
                    } else {
                        k = LB::load_k(u, lane);
                        col = LB::load_col(u, lane) + e;
                    }
                    CHECK(byte >= CF::B_BASE && byte + 4 <= CF::STAGE, "%s byte %d outside the stage", name, byte);
                    CHECK(at.emplace(byte, std::make_tuple(image, col, k)).second, "%s byte %d staged twice", name, byte);
                }
        }
    CHECK((int)at.size() == CF::BN * CF::BK, "%s staged %d of %d elements", name, (int)at.size(), CF::BN * CF::BK);
    for (int n = 0; n < CF::BN; n++)
        for (int k = 0; k < CF::BK; k++) {
            const auto f = at.find(CF::b_elem(k, n));
            CHECK(f != at.end() && f->second == std::make_tuple(n / CF::BH, n % CF::BH, k),
                  "%s element (%d, %d) is not where it is read", name, k, n);
        }
    CHECK(CF::B_BASE >= CF::LA::STAGE, "%s images overlap A", name);
    // Blocks: gate and up at the same columns, every column of a half once.
    std::vector<int> seen(CF::BH, 0);
    for (int wn = 0; wn < CF::WAVES_N; wn++)
        for (int nb = 0; nb < CF::NBH; nb++)
            for (int j = 0; j < CF::BLK; j++) {
                const int c = CF::b_col(wn, nb, j);
                CHECK(c >= 0 && c < CF::BH, "%s gate column %d", name, c);
                if (c >= 0 && c < CF::BH) seen[c]++;
                CHECK(CF::b_col(wn, nb + CF::NBH, j) == c + CF::BH, "%s up column of %d", name, c);
            }
    for (int c = 0; c < CF::BH; c++) CHECK(seen[c] == 1, "%s column %d covered %d times", name, c, seen[c]);
    // Interleaved blocks: a lane's two columns of one k adjoin and are aligned.
    if (CF::B_INTERLEAVE)
        for (int h = 0; h < 2; h++)
            for (int j = 0; j < CF::BLK; j++)
                for (int k = 0; k < CF::BK; k++) {
                    const int a = CF::b_elem(k, CF::b_col(0, h * CF::NBH, j)), b = CF::b_elem(k, CF::b_col(0, h * CF::NBH + 1, j));
                    CHECK(b == a + 4 && a % 8 == 0, "%s interleaved pair at k=%d j=%d", name, k, j);
                }
    // The epilogue's pieces: 16 rows x NBH * BLK columns of a wave.
    constexpr int COLS = CF::NBH * CF::BLK, RR = CF::MF16 ? 4 : 8;
    std::set<std::pair<int, int>> piece;
    for (int l = 0; l < 64; l++)
        for (int nb = 0; nb < CF::NBH; nb++)
            for (int r = 0; r < RR; r++) {
                const int row = CF::acc_row(l / CF::BLK, r), col = CF::b_col(0, nb, l % CF::BLK);
                CHECK(row < 16 && col < COLS, "%s epilogue element (%d, %d)", name, row, col);
                CHECK(piece.insert({row, col}).second, "%s epilogue element (%d, %d) twice", name, row, col);
                for (int rg = 0; rg < CF::NREG / RR; rg++)
                    CHECK(CF::acc_row(l / CF::BLK, rg * RR + r) == rg * 16 + row, "%s epilogue rows", name);
            }
    CHECK((int)piece.size() == 16 * COLS, "%s epilogue covers %d of %d", name, (int)piece.size(), 16 * COLS);
    for (int wn = 0; wn < CF::WAVES_N; wn++)
        for (int nb = 0; nb < CF::NBH; nb++)
            for (int j = 0; j < CF::BLK; j++)
                CHECK(CF::b_col(wn, nb, j) == wn * CF::TN * 16 + CF::b_col(0, nb, j), "%s wave's columns", name);
    printf("%-44s BM x BH = %3d x %-3d LDS = %6d\n", name, CF::BM, CF::BH, CF::LDS_BYTES);
}

#define ONE(wm, wn, tm, tn, bk, v, mf16)                                                          \
    check<Cfg<wm, wn, tm, tn, bk, v, true, true, 2, mf16, true>>(#wm "," #wn "," #tm "," #tn "," #bk "," #v "," #mf16 " F x K"); \
    check<Cfg<wm, wn, tm, tn, bk, v, true, false, 2, mf16, true>>(#wm "," #wn "," #tm "," #tn "," #bk "," #v "," #mf16 " K x F");

int main() {
    ONE(2, 2, 2, 4, 16, true, false)
    ONE(2, 2, 2, 2, 16, true, true)
    ONE(2, 2, 1, 1, 32, true, true)
    ONE(2, 2, 1, 1, 16, false, true)
    ONE(1, 1, 1, 1, 32, true, true)
    ONE(1, 1, 1, 1, 16, false, true)
    printf("failures: %d\n", failures);
    return failures ? 1 : 0;
}
