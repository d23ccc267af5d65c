// The 4-bit output head's kernels for groups of 32 columns.
#include "qs_head_kernels.hpp"

namespace qs {
namespace head {

hipError_t launch_g32(const Args& a, hipStream_t st) { return pick_scale<32>(a, st); }

}  // namespace head
}  // namespace qs
