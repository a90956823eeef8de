#!/bin/bash
# Host-only build of the C ABI of embedding, dropout and log probabilities
# (api_token.cpp) with AddressSanitizer and UndefinedBehaviorSanitizer, linked against launch stubs
# (no GPU code, no HIP runtime).
#   usage: tests/sanitize/build_token.sh OUTPUT
set -e
HERE="$(cd "$(dirname "$0")" && pwd)"
ROOT="$(dirname "$(dirname "$HERE")")"
ROCM="${ROCM_PATH:-/opt/rocm}"
g++ -std=c++17 -O1 -g -fsanitize=address,undefined -fno-sanitize-recover=undefined -fno-omit-frame-pointer \
    -D__HIP_PLATFORM_AMD__ -I"$ROOT/include" -I"$ROOT/collective_communication_reduction_amd/csrc" -I"$HERE" \
    -I"$ROCM/include" \
    "$ROOT/collective_communication_reduction_amd/csrc/api_token.cpp" "$HERE/token_stubs.cpp" "$HERE/token_fuzz.cpp" \
    -o "$1"
