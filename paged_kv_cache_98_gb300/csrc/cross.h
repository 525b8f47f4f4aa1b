// Launchers of cross attention.
#ifndef PKV_CROSS_H
#define PKV_CROSS_H

#include "launch.h"

namespace pkv {

// Cross attention: query rows over an encoder's states (context_lens; max_context bounds
// them).  Work is cut into `ctas` parts; o_part and lse hold two partials of part_rows rows
// for each, cuts what the join needs (all null where no unit can be cut).
struct CrossArgs {
  int max_q;       // bound of the sequences' queries
  int part_rows;   // rows of a partial
  int box_tokens;  // tokens of a query box
  int4* cuts;      // [2 * ctas]: last part, first token, tokens of both query tiles; KV head
};
int launch_cross_d64(const AttnParams& p, const CrossArgs& c, int q_dtype, int kv_dtype, int ctas,
                     cudaStream_t stream);
int launch_cross_d128(const AttnParams& p, const CrossArgs& c, int q_dtype, int kv_dtype, int ctas,
                      cudaStream_t stream);

}  // namespace pkv

#endif  // PKV_CROSS_H
