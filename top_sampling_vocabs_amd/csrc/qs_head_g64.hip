// The 4-bit output head's kernels for groups of 64 columns.
#include "qs_head_kernels.hpp"

namespace qs {
namespace head {

hipError_t launch_g64(const Args& a, hipStream_t st) { return pick_scale<64>(a, st); }

}  // namespace head
}  // namespace qs
