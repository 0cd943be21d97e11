// How dY W of few tokens spreads its contraction, W's rows, over workgroups: a
// workgroup takes a block of columns and one part, a run of rows, in steps. Plain
// C++, so that a program of the host alone can go through it.
#pragma once

constexpr int FP4_CWV = 8;            // waves of a workgroup
constexpr int FP4_CN = 32 * FP4_CWV;  // rows that they take at once, 32 each

struct ColsPlan {
    int parts;
    int per;  // rows of a part: whole steps, so that no step reaches into the next part
    int sets; // sets of CN rows of a step
};

// Parts of the contraction over N rows, of columns in nkb blocks (one at least):
// about a workgroup a CU, a part's rows whole sets. Two sets a step, all of whose
// loads are in flight, where a part is whole steps of them, else one (16 tokens over
// 6144 x 4096, 8 parts of three sets: 10.6 us; parts of four sets in two steps, 6 of
// them, 11.2; three sets in two steps, the second half empty, 11.9).
inline ColsPlan cols_plan(int N, int nkb)
{
    const int all = (N + FP4_CN - 1) / FP4_CN, want = nkb < 256 ? 256 / nkb : 1;
    const int most = all < want ? all : want;
    if (most == 0)
        return {1, FP4_CN, 1};
    const int run = (N + most - 1) / most, per = (run + FP4_CN - 1) / FP4_CN * FP4_CN;
    return {(N + per - 1) / per, per, per % (2 * FP4_CN) == 0 ? 2 : 1};
}
