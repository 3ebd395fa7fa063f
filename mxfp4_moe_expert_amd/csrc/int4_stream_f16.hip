// int4_stream_f16.hip -- the streaming int4 kernels for fp16 activations.
#include "int4_stream.h"

namespace k3g {
int launch_int4_stream_f16(const I4Args &a, int mode, int group, int form, hipStream_t st) {
    return launch_int4_stream_type<K3G_F16>(a, mode, group, form, st);
}
}  // namespace k3g
