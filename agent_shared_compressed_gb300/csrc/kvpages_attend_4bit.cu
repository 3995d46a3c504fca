// kvpages_attend_4bit.cu -- attention over pages with 4-bit keys (kvpages_attend.cuh),
// with and without a window.
#include "kvpages_attend.cuh"

namespace kvp {

template int launch_attend<128, KVP_PAGES_K4V4, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_K4V4, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<128, KVP_PAGES_K4V4, true>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_K4V4, true>(PagesAttendArgs &, int, cudaStream_t);

}  // namespace kvp
