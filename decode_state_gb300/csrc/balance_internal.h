// Between balance.cu and the translation units with the kernels over rows of each type of logits.
#pragma once

#include <stddef.h>

namespace sdm {

// A kernel over rows: its threads, the rows that a block works on at a time, its dynamic shared memory.
struct BalanceTeam {
    const void* fn;
    int threads, teams;
    size_t smem;
};

// For rows of n entries; vec: rows of 16-byte pieces; grad: with the gradient.
BalanceTeam balance_team_bf16(int n, bool vec, bool grad);
BalanceTeam balance_team_f32(int n, bool vec, bool grad);

}  // namespace sdm
