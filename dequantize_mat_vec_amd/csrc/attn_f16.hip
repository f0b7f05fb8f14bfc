// Paged attention over binary16 pages (kernel in attn_impl.h).
#include "attn_impl.h"

namespace pesti_attn {
int launch_f16(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) { return launch_format<false>(p, rows, st); }
}  // namespace pesti_attn
