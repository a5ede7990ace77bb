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
  {  // a list is of the device it was made on
    float data[4] = {}, norm = 0, one = 1;
    const void* ptr[1] = {data};
    const size_t count[1] = {4};
    int32_t workspace[8] = {};
    hocTensorList_t *here = nullptr, *there = nullptr;
    fake::device = 1;
    CHECK(hoc_tensor_list_create(&there, 1, ptr, count, HOC_FLOAT32) == HOC_SUCCESS);
    fake::device = 0;
    CHECK(hoc_tensor_list_create(&here, 1, ptr, count, HOC_FLOAT32) == HOC_SUCCESS);
    CHECK(hoc_grad_norm(there, &norm, workspace, 8, nullptr) == HOC_ERR_INVALID_ARG);
    CHECK(hoc_grad_clip(there, there, &one, &norm, workspace, 8, nullptr) == HOC_ERR_INVALID_ARG);
    CHECK(hoc_grad_clip(here, there, &one, &norm, workspace, 8, nullptr) == HOC_ERR_INVALID_ARG);
    CHECK(hoc_grad_clip(there, here, &one, &norm, workspace, 8, nullptr) == HOC_ERR_INVALID_ARG);
    CHECK(fake::launches == 0);
    CHECK(hoc_grad_norm(here, &norm, workspace, 8, nullptr) == HOC_SUCCESS);
    CHECK(hoc_grad_clip(here, here, &one, &norm, workspace, 8, nullptr) == HOC_SUCCESS);
    CHECK(fake::launches == 4);
    fake::device = 1;
    CHECK(hoc_grad_norm(there, &norm, workspace, 8, nullptr) == HOC_SUCCESS);
    fake::device = 0;
    fake::refuse = true;  // a failed launch is reported, and leaves no error for the next call
    CHECK(hoc_grad_norm(here, &norm, workspace, 8, nullptr) == HOC_ERR_CUDA && fake::last == 0);
    CHECK(hoc_grad_clip(here, here, &one, &norm, workspace, 8, nullptr) == HOC_ERR_CUDA && fake::last == 0);
    fake::refuse = false;
    CHECK(hoc_tensor_list_destroy(there) == HOC_SUCCESS && hoc_tensor_list_destroy(here) == HOC_SUCCESS);
  }
  printf("LISTS OK\n");
  return 0;
}
