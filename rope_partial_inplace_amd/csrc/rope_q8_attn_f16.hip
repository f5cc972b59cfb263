// rope_q8_attn_f16.hip -- attention over a paged cache in 8 bits for float16 queries.
#include "rope_q8_rows.h"

namespace ropeamd {

int run_attention_q8_f16(AttnQ8Plan &p, void *stream) { return run_attention_q8<_Float16>(p, stream); }

}  // namespace ropeamd
