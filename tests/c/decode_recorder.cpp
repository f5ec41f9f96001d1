// The launches of the decode-step operators, recorded instead of made: linked with
// decode.cpp and plan.cpp in place of the device code, so that tests see which
// calls are accepted, and with what, on a host without a device.
#include "decode.h"
#include "internal.h"

namespace detfold_impl {

static int launches, width;
int launch_append(const AppendArgs &a, void *) { return ++launches, width = a.width, DETFOLD_OK; }
int launch_softmax(const SoftmaxArgs &, void *) { return ++launches, DETFOLD_OK; }
int launch_attend(const AttendArgs &, void *) { return ++launches, DETFOLD_OK; }
int current_cu_count(int32_t *cu) { return *cu = 256, DETFOLD_OK; }

}  // namespace detfold_impl

extern "C" int recorded_launches() { return detfold_impl::launches; }
extern "C" int recorded_width() { return detfold_impl::width; }  // of the last append
