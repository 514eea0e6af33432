// The balance loss over float32 logits.
#include "balance_rows.cuh"

namespace sdm {

BalanceTeam balance_team_f32(int n, bool vec, bool grad) { return rows_team<float>(n, vec, grad); }

}  // namespace sdm
