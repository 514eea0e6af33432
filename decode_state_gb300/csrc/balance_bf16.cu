// The balance loss over bfloat16 logits.
#include "balance_rows.cuh"

namespace sdm {

BalanceTeam balance_team_bf16(int n, bool vec, bool grad) { return rows_team<uint16_t>(n, vec, grad); }

}  // namespace sdm
