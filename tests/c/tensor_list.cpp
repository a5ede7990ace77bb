// Tensor lists of csrc/grad.cu over the fake runtime.
#include <cstdio>
#include <vector>

#include "fake_cudart.h"
#include "hoc_grad.h"

namespace hoc {
void set_error_detail(const char*) {}
}  // namespace hoc

#define CHECK(cond)                                          \
  do {                                                       \
    if (!(cond)) {                                           \
      printf("FAIL %s:%d: %s\n", __FILE__, __LINE__, #cond); \
      return 1;                                              \
    }                                                        \
  } while (0)

int main() {
  for (int n : {1, 3, 5000}) {  // tables of 16 bytes to more than 64 KB
    std::vector<float> data(n);
    std::vector<const void*> ptr(n);
    std::vector<size_t> count(n, 1);
    for (int i = 0; i < n; ++i) ptr[i] = &data[i];
    hocTensorList_t* list = nullptr;
    CHECK(hoc_tensor_list_create(&list, n, ptr.data(), count.data(), HOC_FLOAT32) == HOC_SUCCESS);
    CHECK(fake::copies_under_way() == 0);  // the table is on the device
    CHECK(hoc_tensor_list_destroy(list) == HOC_SUCCESS);
  }
  printf("LISTS OK\n");
  return 0;
}
