#pragma once
namespace fake {
extern int device;     // the current one, of two
extern int launches;   // of kernels, so far
extern int last;       // error that has not been read, 0: none
extern unsigned widest;  // most CTAs along x of a launch, so far
extern bool refuse;    // every launch
int copies_under_way();  // from the host, not yet on the device
}  // namespace fake
