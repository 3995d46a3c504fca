// kvpages_attend_window.cu -- attention over pages with a window and first tokens
// (kvpages_attend.cuh), for all formats but 4-bit keys.
#include "kvpages_attend.cuh"

namespace kvp {

template int launch_attend<128, KVP_PAGES_BF16, true>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_BF16, true>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<128, KVP_PAGES_K8V8, true>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_K8V8, true>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<128, KVP_PAGES_K8V4, true>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_K8V4, true>(PagesAttendArgs &, int, cudaStream_t);

}  // namespace kvp
