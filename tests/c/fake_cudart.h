#pragma once
namespace fake {
extern int device;     // the current one, of two
extern int launches;   // of kernels, so far
int copies_under_way();  // from the host, not yet on the device
}  // namespace fake
