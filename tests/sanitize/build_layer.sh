#!/bin/bash
# Host-only build of the layer operators' C ABI (api_layer.cpp) with
# AddressSanitizer and UndefinedBehaviorSanitizer, linked against launch stubs
# (no GPU code, no HIP runtime).
#   usage: tests/sanitize/build_layer.sh OUTPUT
set -e
HERE="$(cd "$(dirname "$0")" && pwd)"
ROOT="$(dirname "$(dirname "$HERE")")"
ROCM="${ROCM_PATH:-/opt/rocm}"
g++ -std=c++17 -O1 -g -fsanitize=address,undefined -fno-sanitize-recover=undefined -fno-omit-frame-pointer \
    -D__HIP_PLATFORM_AMD__ -I"$ROOT/include" -I"$ROOT/collective_communication_reduction_amd/csrc" -I"$HERE" \
    -I"$ROCM/include" \
    "$ROOT/collective_communication_reduction_amd/csrc/api_layer.cpp" "$HERE/layer_stubs.cpp" "$HERE/layer_fuzz.cpp" \
    -o "$1"
