#!/bin/bash
# Builds grouped_driver.cpp (which see) with the address and undefined-behaviour sanitizers in the
# host code into the file named by $1.  No GPU and no built library needed.
set -e
HERE=$(cd "$(dirname "$0")" && pwd)
R=$(cd "$HERE/../.." && pwd)
/opt/rocm/bin/hipcc -O1 -g -std=c++17 --offload-arch=gfx950 -Wall -I "$R/include" -I "$R/tiled_matrix_multiply_amd/csrc" \
  -Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined -Xarch_host -fno-omit-frame-pointer \
  -c "$HERE/grouped_driver.cpp" -o "$1.o"
/opt/rocm/llvm/bin/clang++ -fsanitize=address -fsanitize=undefined "$1.o" -L/opt/rocm/lib -lamdhip64 -Wl,-rpath,/opt/rocm/lib -o "$1"
