// fa_kv4_status.h -- the status word of the cache kernels (fa_kv4.cu), for
// the calls that report the device status (fa_api.cu).  Not exported.
#pragma once

#include "fa_gb300.h"

#define FA_LOCAL __attribute__((visibility("hidden")))
// Reads (and clears, if asked) the word of the current device.
FA_LOCAL int fa_kv4_status_read(int clear, int* value);
// Reads it in the order of `stream`; *value holds it once the stream has been waited for.
FA_LOCAL int fa_kv4_status_read_async(int* value, fa_stream_t stream);
