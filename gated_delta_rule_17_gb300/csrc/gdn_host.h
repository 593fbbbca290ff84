// What the library's translation units share on the host: the calling thread's error message and launch
// count, the device's status word, and the TMA encoder. Defined in gdn_api.cu.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#pragma GCC visibility push(hidden)
namespace gdn_host {
void begin();                                 // a call begins: no error, no launches
int refuse(int code, const char* message);    // sets the error message; returns code
void count(int launches);
int device(int* sms, unsigned** status);      // of the current device, or the error's code
int plan_sms();                               // SMs to plan by, also where there is no device
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}  // namespace gdn_host
#pragma GCC visibility pop
