// Paged attention over 8-bit pages with a scale per row (kernel in attn_impl.h).
#include "attn_impl.h"

namespace pesti_attn {
int launch_i8(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) { return launch_format<true>(p, rows, st); }
}  // namespace pesti_attn
